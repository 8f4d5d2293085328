// Tokens sorted by the experts they were routed to, and back.
//
// Sorting is a counting sort that keeps the order of equal ones: place s =
// t k + j goes behind all places of smaller experts and the earlier ones of its
// own.  Places without an expert stand behind all, so that every row of the
// result has one place, and those rows are zeros.  All of it is bound by the
// rows moved: tokens are walked in order, each row of x is read and each of y
// written once (dy once for each four of a token's places), and the rows by expert once.
//
// One GB300, inputs changing between calls: dispatch of 8192 x 8 rows of 2048
// bf16 (302 MB) 52.6 us, 5.7 TB/s: the rows 44 us, counts and ranks before them
// the rest (68 us with 384 experts, 69.5 with 512, whose ranks go a warp after another);
// combine of them 48.7 us, 6.2 TB/s; their gradients (571 MB, dy once more than that) 100.6 us; the
// gradients of 4093 x 6 rows of 1001 f32, none on a
// 16-byte boundary, 46.5 us (a 213 MB case whose scalar loads and stores bound it).
// 16 x 4 rows of 4096 bf16 are dispatched in 2.4 us of a graph by one launch.
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

constexpr int kThreads = 256;
// (1024 threads that rank: dispatch of 65536 places 52.5 us in a graph, 56 with 512)
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kByWarp = 320;       // experts (and one) that are counted by warp: as many as 48 KB hold
static_assert((2 + kSortWarps) * kByWarp * sizeof(unsigned) < 48 * 1024 - 256, "the counts fit without more being asked for");
constexpr int kFewPlaces = 1024;   // places that every block ranks for itself

// The expert of place s; `experts` where it has none.
__device__ __forceinline__ int expert_of(const int64_t* idx, int64_t s, int experts) {
  const int64_t v = idx[s];
  return v >= 0 && v < experts ? static_cast<int>(v) : experts;
}

// ---- ranks ------------------------------------------------------------------------
// counts[b * (experts + 1) + e]: places of expert e in block b's run of `chunk` places.
__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const int64_t* idx, int64_t total, int64_t chunk, int experts,
                                                                    unsigned* counts) {
  extern __shared__ unsigned held[];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int e = threadIdx.x; e <= experts; e += kSortThreads) held[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * chunk, end = min(begin + chunk, total);
  for (int64_t s = begin + threadIdx.x; s < end; s += kSortThreads) atomicAdd(&held[expert_of(idx, s, experts)], 1u);
  __syncthreads();
  for (int e = threadIdx.x; e <= experts; e += kSortThreads) counts[int64_t(blockIdx.x) * (experts + 1) + e] = held[e];
}

// Row of every place: rows[s], or ~row of the zeros for a place without an expert.
__global__ void __launch_bounds__(kSortThreads) expert_rank_kernel(const int64_t* idx, int64_t total, int64_t chunk, int experts,
                                                                   const unsigned* counts, int* rows, int64_t* place, int64_t* offsets) {
  extern __shared__ unsigned held[];
  __shared__ unsigned warp_sum[kSortWarps];
  unsigned* all = held;                  // places of each expert, then where the next place of this block goes
  unsigned* before = held + experts + 1; // those of the blocks before
  grid_dependency_wait();
  grid_launch_dependents();
  const int kinds = experts + 1;
  for (int e = threadIdx.x; e < 2 * kinds; e += kSortThreads) held[e] = 0;
  __syncthreads();
  // a thread adds up some of the blocks' counts of one expert, eight of them under way
  const int across = min(kinds, kSortThreads), groups = kSortThreads / across, blocks = static_cast<int>(gridDim.x);
  if (static_cast<int>(threadIdx.x) < groups * across) {
    for (int e = threadIdx.x % across; e < kinds; e += across) {
      unsigned sum = 0, earlier = 0;
      for (int b0 = threadIdx.x / across; b0 < blocks; b0 += 8 * groups) {
        unsigned v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = b0 + q * groups < blocks ? counts[(b0 + q * groups) * kinds + e] : 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          sum += v[q];
          if (b0 + q * groups < static_cast<int>(blockIdx.x)) earlier += v[q];
        }
      }
      if (sum) atomicAdd(&all[e], sum);
      if (earlier) atomicAdd(&before[e], earlier);
    }
  }
  __syncthreads();
  // bases by a scan over the experts, a run of them a thread
  const int run = (kinds + kSortThreads - 1) / kSortThreads;
  const int e0 = min(kinds, static_cast<int>(threadIdx.x) * run), e1 = min(kinds, e0 + run);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  unsigned sum = 0;
  for (int e = e0; e < e1; ++e) sum += all[e];
  unsigned incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  unsigned base = incl - sum;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  for (int e = e0; e < e1; ++e) {
    const unsigned n = all[e];
    if (blockIdx.x == 0) offsets[e] = base;  // (offsets[experts]: the start of those without an expert)
    all[e] = base + before[e];
    base += n;
  }
  __syncthreads();
  // the block's places in order, kSortThreads at a time
  const int64_t begin = blockIdx.x * chunk, end = min(begin + chunk, total);
  unsigned* by_warp = before + kinds;    // places of each expert in each warp, where there is room for them
  for (int64_t s0 = begin; s0 < end; s0 += kSortThreads) {
    const int64_t s = s0 + threadIdx.x;
    const int e = s < end ? expert_of(idx, s, experts) : -1;
    unsigned row = 0;
    if (kinds <= kByWarp) {
      for (int i = threadIdx.x; i < kSortWarps * kinds; i += kSortThreads) by_warp[i] = 0;
      __syncthreads();
      const unsigned same = __match_any_sync(~0u, e);
      if (e >= 0 && (same & lanemask_lt()) == 0) by_warp[warp * kinds + e] = __popc(same);
      __syncthreads();
      for (int i = threadIdx.x; i < kinds; i += kSortThreads) {
        unsigned at = all[i];
        for (int w = 0; w < kSortWarps; ++w) {
          const unsigned n = by_warp[w * kinds + i];
          by_warp[w * kinds + i] = at;
          at += n;
        }
        all[i] = at;
      }
      __syncthreads();
      if (e >= 0) row = by_warp[warp * kinds + e] + __popc(same & lanemask_lt());
    } else {  // a warp after another
      for (int w = 0; w < kSortWarps; ++w) {
        if (w == warp) {
          const unsigned same = __match_any_sync(~0u, e);
          if (e >= 0) {
            row = all[e] + __popc(same & lanemask_lt());
            __syncwarp(same);
            if ((same & lanemask_lt()) == 0) all[e] += __popc(same);
          }
        }
        __syncthreads();
      }
    }
    if (e >= 0) {
      rows[s] = e < experts ? static_cast<int>(row) : ~static_cast<int>(row);
      place[s] = e < experts ? static_cast<int64_t>(row) : -1;
    }
    __syncthreads();
  }
}

// ---- moving rows --------------------------------------------------------------------
// What one of `share` threads (whole warps) holds of a row of d values: 16 bytes side by side where rows allow it, else
// SCALARS values 32 apart, so that as many bytes are under way and a warp's loads are whole lines all the same.
template <typename T, int VEC, int SCALARS = 16 / static_cast<int>(sizeof(T))>
struct Piece {
  static constexpr int kWide = VEC > 1 ? VEC : SCALARS;
  Raw<T, VEC> r[VEC > 1 ? 1 : kWide];
  __device__ __forceinline__ static int first(int at) { return VEC > 1 ? at * VEC : at / 32 * (32 * kWide) + at % 32; }
  __device__ __forceinline__ static int step(int share) { return share * kWide; }
  __device__ __forceinline__ void load(const T* row, int c, int d) {
    if constexpr (VEC > 1) {
      r[0].load_nc(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < kWide; ++e) {
        r[e].clear();
        if (c + e * 32 < d) r[e].load_nc(row + c + e * 32);
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (auto& v : r) v.clear();
  }
  __device__ __forceinline__ void values(float* f) const {
    if constexpr (VEC > 1) {
      Vec<T, VEC> v;
      v.set_raw(r[0]);
#pragma unroll
      for (int e = 0; e < kWide; ++e) f[e] = v.v[e];
    } else {
#pragma unroll
      for (int e = 0; e < kWide; ++e) f[e] = to_f32(r[e].u);
    }
  }
  __device__ __forceinline__ void store(T* row, int c, int d) const {
    if constexpr (VEC > 1) {
      __stcs(reinterpret_cast<uint4*>(row + c), r[0].u);
    } else {
#pragma unroll
      for (int e = 0; e < kWide; ++e)
        if (c + e * 32 < d) row[c + e * 32] = r[e].u;
    }
  }
  __device__ __forceinline__ static void store(const float* f, T* row, int c, int d) {
    if constexpr (VEC > 1) {
      Vec<T, VEC> v;
#pragma unroll
      for (int e = 0; e < kWide; ++e) v.v[e] = f[e];
      v.store_stream(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < kWide; ++e)
        if (c + e * 32 < d) row[c + e * 32] = from_f32<T>(f[e]);
    }
  }
};

struct MoveRows {
  const void* x;
  int64_t ldx, tokens, d;
  int k, experts;
  const int64_t* idx;
  int64_t* place;
  int64_t* offsets;
  const int* rows;
  void* xs;
};

// Writes token t's row to the k rows of its places (zeros to those without an expert), `share` threads of which this is `at`.
template <typename T, int VEC>
__device__ __forceinline__ void spread_row(const MoveRows& p, int64_t t, const int* rows, int at, int share) {
  using P = Piece<T, VEC>;
  const int d = static_cast<int>(p.d);
  const T* src = static_cast<const T*>(p.x) + t * p.ldx;
  for (int c = P::first(at); c < d; c += P::step(share)) {
    P v, zero;
    v.load(src, c, d);
    zero.clear();
    for (int j = 0; j < p.k; ++j) {
      const int r = rows[j];
      T* dst = static_cast<T*>(p.xs) + static_cast<int64_t>(r < 0 ? ~r : r) * p.d;
      if (r < 0) zero.store(dst, c, d);
      else v.store(dst, c, d);
    }
  }
}

// Few places: block t ranks token t's places by counting those that stand before them and moves its row; the last block forms
// the offsets.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) dispatch_few_kernel(const MoveRows p) {
  __shared__ int rows[kFewPlaces];
  extern __shared__ unsigned held[];
  grid_dependency_wait();
  grid_launch_dependents();
  const int total = static_cast<int>(p.tokens) * p.k;
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (t == p.tokens) {
    const int kinds = p.experts + 1;
    for (int e = threadIdx.x; e < kinds; e += kThreads) held[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < total; s += kThreads) atomicAdd(&held[expert_of(p.idx, s, p.experts)], 1u);
    __syncthreads();
    if (warp == 0) {
      unsigned base = 0;
      for (int e0 = 0; e0 < kinds; e0 += 32) {
        const unsigned n = e0 + lane < kinds ? held[e0 + lane] : 0;
        unsigned incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned v = __shfl_up_sync(~0u, incl, o);
          if (lane >= o) incl += v;
        }
        if (e0 + lane < kinds) p.offsets[e0 + lane] = base + incl - n;
        base += __shfl_sync(~0u, incl, 31);
      }
    }
    return;
  }
  for (int j = warp; j < p.k; j += kThreads / 32) {
    const int s = static_cast<int>(t) * p.k + j;
    const int e = expert_of(p.idx, s, p.experts);
    int row = 0;
    for (int i = lane; i < total; i += 32) {
      const int other = expert_of(p.idx, i, p.experts);
      row += other < e || (other == e && i < s);
    }
    row = __reduce_add_sync(~0u, row);
    if (lane == 0) {
      rows[j] = e < p.experts ? row : ~row;
      p.place[s] = e < p.experts ? row : -1;
    }
  }
  __syncthreads();
  spread_row<T, VEC>(p, t, rows, threadIdx.x, kThreads);
}

// `share` threads a token (a power of two).
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const MoveRows p, int share) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = int64_t(blockIdx.x) * (kThreads / share) + threadIdx.x / share;
  if (t < p.tokens) spread_row<T, VEC>(p, t, p.rows + t * p.k, threadIdx.x % share, share);
}

// ---- back ---------------------------------------------------------------------------
struct JoinRows {
  const void* ys;
  int64_t ldy, rows, tokens, d;
  int k;
  const int64_t* place;
  const void* weights;  // nullable
  void* y;
  const void* dy;       // gradients: of y
  int64_t lddy;
  unsigned* listed;     // how often each row is listed,
  int *first, *last, *next;  // one of its places, and a chain of the others, in no order: one of them, and from each the next
  void* dys;            // nullable
  void* dweights;       // nullable
};
constexpr int kRowsTogether = 4;  // rows of a token that are read together
constexpr int kRowsBlock = 32; // rows that a block of rows looks after
constexpr int kChain = 128;    // places of a row that a warp ranks (256, of 8 KB a block: 68 us instead of 65 for 4093 x 6 rows of 2001 bf16)

// What a token's places hold: their rows (-1: none) and weights, kTogether of them from the j0-th on.
template <typename T, int kTogether>
struct Listed {
  int row[kTogether];
  float f[kTogether];
  __device__ __forceinline__ void load(const JoinRows& p, int64_t t, int j0) {
    const int64_t* place = p.place + t * p.k + j0;
    const T* w = static_cast<const T*>(p.weights) + t * p.k + j0;
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const bool in = t < p.tokens && j0 + j < p.k;
      const int64_t r = in ? place[j] : -1;
      row[j] = r >= 0 && r < p.rows ? static_cast<int>(r) : -1;
      f[j] = row[j] < 0 ? 0.0f : p.weights ? to_f32(w[j]) : 1.0f;
    }
  }
};

// (Blocks that take several tokens in turn, the next one's places loaded ahead, have 97 registers instead of 72: 58 us instead
// of 54, before a thread took two pieces, for 8192 x 8 rows of 2048 bf16.)
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const JoinRows p, int share) {
  using P = Piece<T, VEC>;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = int64_t(blockIdx.x) * (kThreads / share) + threadIdx.x / share;
  if (t >= p.tokens) return;
  constexpr int kTogether = kRowsTogether;
  const T* ys = static_cast<const T*>(p.ys);
  const T* w = static_cast<const T*>(p.weights) + (p.weights ? t * p.k : 0);
  const int64_t* place = p.place + t * p.k;
  const int d = static_cast<int>(p.d);
  for (int c = P::first(threadIdx.x % share); c < d; c += P::step(share)) {
    float sum[P::kWide] = {};
    for (int j0 = 0; j0 < p.k; j0 += kTogether) {
      P v[kTogether];
      float f[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        const int64_t r = j0 + j < p.k ? place[j0 + j] : -1;
        f[j] = 0.0f;
        if (r >= 0 && r < p.rows) {
          v[j].load(ys + r * p.ldy, c, d);
          f[j] = p.weights ? to_f32(w[j0 + j]) : 1.0f;
        } else {
          v[j].clear();
        }
      }
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        float x[P::kWide];
        v[j].values(x);
#pragma unroll
        for (int e = 0; e < P::kWide; ++e) sum[e] = fmaf(f[j], x[e], sum[e]);
      }
    }
    P::store(sum, static_cast<T*>(p.y) + t * p.d, c, d);
  }
}

__global__ void __launch_bounds__(kThreads) clear_listed_kernel(unsigned* listed, int64_t rows) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t r = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (r < rows) listed[r] = 0;
}
__global__ void __launch_bounds__(kThreads) count_listed_kernel(const int64_t* place, int64_t total, unsigned* listed, int* first, int* last, int* next,
                                                                int64_t rows) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t s = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (s >= total) return;
  const int64_t r = place[s];
  if (r < 0 || r >= rows) return;
  // (a chain's end is what `last` held before: it is walked by its length)
  if (atomicAdd(&listed[r], 1u) == 0) first[r] = static_cast<int>(s);
  else next[s] = atomicExch(&last[r], static_cast<int>(s));
}

// A warp: the sum of row r, which `times` (2 or more) places list, in their order.  The chain's order is the atomics', so the places
// are ranked first.  (By value: with the kernel's parameters handed down by their address all of it read them from memory.)
template <typename T, int VEC>
__device__ __noinline__ void sum_chain(const int* next, int first, int last, int times, int k, const T* dy, int64_t lddy, const T* weights,
                                       int d, T* dst, int* places) {
  using P = Piece<T, VEC, 4>;
  const int lane = threadIdx.x % 32;
  if (lane == 0) {
    places[0] = first;
    int s = last;
    for (int i = 1;; s = next[s]) {
      places[i] = s;
      if (++i == times) break;
    }
  }
  __syncwarp();
  int held[kChain / 32], rank[kChain / 32];
#pragma unroll
  for (int e = 0; e < kChain / 32; ++e) {
    held[e] = e * 32 + lane < times ? places[e * 32 + lane] : 0;
    rank[e] = 0;
  }
  for (int i = 0; i < times; ++i) {
    const int other = places[i];
#pragma unroll
    for (int e = 0; e < kChain / 32; ++e) rank[e] += other < held[e];
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < kChain / 32; ++e)
    if (e * 32 + lane < times) places[rank[e]] = held[e];
  __syncwarp();
  for (int c = P::first(lane); c < d; c += P::step(32)) {
    float sum[P::kWide] = {};
    for (int i = 0; i < times; ++i) {
      const int s = places[i];
      const float f = weights ? to_f32(weights[s]) : 1.0f;
      P raw;
      raw.load(dy + int64_t(s / k) * lddy, c, d);
      float g[P::kWide];
      raw.values(g);
#pragma unroll
      for (int e = 0; e < P::kWide; ++e) sum[e] = fmaf(f, g[e], sum[e]);
    }
    P::store(sum, dst, c, d);
  }
  __syncwarp();
}

// Four rows of a token together: with eight, 128 registers left 16 warps an SM (with one piece a thread 136 us instead of 120 for
// 8192 x 8 rows of 2048 bf16, 59 instead of 52 for the odd f32 ones); with two, 133 and 52.
//
// Blocks of tokens, `share` threads each (32 or more): what a place's row gets where no other place lists it, and the products
// that are the weights' gradients.  Behind them blocks of rows: zeros for rows that no place lists, and the sums, in order
// of place, for rows that more than one does (permutations have none): by a warp from the row's chain, or, where more than kChain
// do, by the block from a scan over all places, which only that few rows can take.  (With the scan for
// all, 32768 rows of 512 f32 that 65536 places list twice took 7.2 ms, and four times that for each doubling: minutes for
// 2^24 places.)
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const JoinRows p, int share, int64_t token_blocks) {
  constexpr int kTogether = kRowsTogether;
  __shared__ float dots[kThreads / 32][kTogether];
  __shared__ unsigned listed[kRowsBlock];
  __shared__ unsigned hit_mask[kThreads / 32];
  __shared__ int places[kThreads / 32][kChain];
  grid_dependency_wait();
  grid_launch_dependents();
  const T* ys = static_cast<const T*>(p.ys);
  const T* dy = static_cast<const T*>(p.dy);
  const T* weights = static_cast<const T*>(p.weights);
  T* dys = static_cast<T*>(p.dys);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  using P = Piece<T, VEC, 4>;  // (eight bf16 values: 84 us instead of 74, before a thread took four pieces, for 4093 x 6 rows of 2001)
  const int d = static_cast<int>(p.d);
  if (blockIdx.x < token_blocks) {
    // (in turn, a token's places loaded while the one before is worked on)
    const int at = threadIdx.x % share, each = kThreads / share;
    const int64_t step = token_blocks * each, rounds = (p.tokens + step - 1) / step;
    int64_t t = int64_t(blockIdx.x) * each + threadIdx.x / share;
    Listed<T, kTogether> next;
    next.load(p, t, 0);
    for (int64_t round = 0; round < rounds; ++round, t += step) {
      Listed<T, kTogether> now = next;
      const bool in = t < p.tokens;
      for (int j0 = 0; j0 < p.k; j0 += kTogether) {
        if (j0) now.load(p, t, j0);
        unsigned times[kTogether];
        float dot[kTogether] = {};
#pragma unroll
        for (int j = 0; j < kTogether; ++j) times[j] = dys && now.row[j] >= 0 ? p.listed[now.row[j]] : 0;
        for (int c = P::first(at); in && c < d; c += P::step(share)) {
          P raw, v[kTogether];
          raw.load(dy + t * p.lddy, c, d);
          if (p.dweights) {
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
              if (now.row[j] >= 0) v[j].load(ys + now.row[j] * p.ldy, c, d);
          }
          if (j0 == 0 && c == P::first(at)) next.load(p, t + step, 0);
          float g[P::kWide];
          raw.values(g);
#pragma unroll
          for (int j = 0; j < kTogether; ++j) {
            if (now.row[j] < 0) continue;
            float x[P::kWide];
            if (times[j] == 1) {
#pragma unroll
              for (int e = 0; e < P::kWide; ++e) x[e] = now.f[j] * g[e];
              P::store(x, dys + now.row[j] * p.d, c, d);
            }
            if (p.dweights) {
              v[j].values(x);
#pragma unroll
              for (int e = 0; e < P::kWide; ++e) dot[j] = fmaf(x[e], g[e], dot[j]);
            }
          }
        }
        if (!p.dweights) continue;
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
#pragma unroll
          for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(~0u, dot[j], o);
          if (lane == 0) dots[warp][j] = dot[j];
        }
        __syncthreads();
        if (in && at < kTogether && j0 + at < p.k) {
          float sum = 0.0f;
          for (int w = 0; w < share / 32; ++w) sum += dots[warp + w][at];
          static_cast<T*>(p.dweights)[t * p.k + j0 + at] = from_f32<T>(sum);
        }
        __syncthreads();
      }
    }
    return;
  }
  const int64_t r0 = (int64_t(blockIdx.x) - token_blocks) * kRowsBlock;
  unsigned mine = 1;
  if (threadIdx.x < kRowsBlock) listed[threadIdx.x] = mine = r0 + threadIdx.x < p.rows ? p.listed[r0 + threadIdx.x] : 1;
  const bool shared = __syncthreads_or(mine > 1);
  P zero;
  zero.clear();
  for (int q = warp; q < kRowsBlock; q += kThreads / 32)
    if (listed[q] == 0)
      for (int c = P::first(lane); c < d; c += P::step(32)) zero.store(dys + (r0 + q) * p.d, c, d);
  if (!shared) return;  // (asked of the block at once: with the question by row, and a call behind it, 46 us instead of 31 for 16384 x 8 rows of 64)
#pragma unroll 1
  for (int q = warp; q < kRowsBlock; q += kThreads / 32) {
    if (listed[q] > 1 && listed[q] <= kChain) {
      const int64_t r = r0 + q;
      sum_chain<T, VEC>(p.next, p.first[r], p.last[r], static_cast<int>(listed[q]), p.k, dy, p.lddy, weights, d, dys + r * p.d, places[warp]);
    }
  }
  const int64_t total = p.tokens * p.k;
  for (int q = 0; q < kRowsBlock; ++q) {
    const unsigned times = listed[q];
    if (times <= kChain) continue;
    const int64_t r = r0 + q;
    for (int64_t c0 = 0; c0 < p.d; c0 += kThreads * VEC) {
      const int64_t c = c0 + threadIdx.x * VEC;
      Vec<T, VEC> sum;
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum.v[e] = 0.0f;
      unsigned seen = 0;
      for (int64_t s0 = 0; seen < times && s0 < total; s0 += kThreads) {
        const bool hit = s0 + threadIdx.x < total && p.place[s0 + threadIdx.x] == r;
        const unsigned hits = __ballot_sync(~0u, hit);
        __syncthreads();
        if (lane == 0) hit_mask[warp] = hits;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w)
          for (unsigned m = hit_mask[w]; m; m &= m - 1) {
            const int64_t s = s0 + w * 32 + __ffs(static_cast<int>(m)) - 1;
            ++seen;
            if (c >= p.d) continue;
            const float f = weights ? to_f32(weights[s]) : 1.0f;
            Vec<T, VEC> g;
            g.load_nc(dy + s / p.k * p.lddy + c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum.v[e] = fmaf(f, g.v[e], sum.v[e]);
          }
      }
      if (c < p.d) sum.store_stream(dys + r * p.d + c);
    }
  }
}

// Whether rows can be read and written 16 bytes at a time.
bool whole_vectors(int64_t size, int64_t d, std::initializer_list<const void*> at, std::initializer_list<int64_t> lds) {
  uintptr_t low = static_cast<uintptr_t>(d * size);
  for (const void* p : at) low |= reinterpret_cast<uintptr_t>(p);
  for (int64_t ld : lds) low |= static_cast<uintptr_t>(ld * size);
  return low % 16 == 0;
}
// Threads that share a token's row: a power of two, one piece each or more, a warp at least.
int share_of(int64_t d, int wide) {
  int share = 32;
  while (share < kThreads && int64_t(share) * wide < d) share *= 2;
  return share;
}
int64_t blocks_of(int64_t tokens, int share) { return (tokens + kThreads / share - 1) / (kThreads / share); }
// As many of them as fit at once, so that each takes several tokens.
template <typename K>
cudaError_t blocks_at_once(K kernel, PerDevice& known, int64_t* blocks) {
  std::atomic<int>* k = known.here();
  int each = k ? k->load() : 0;
  if (!each) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, kThreads, 0);
    if (e != cudaSuccess) return e;
    if (each < 1) each = 1;
    if (k) *k = each;
  }
  const int64_t most = int64_t(each) * ops_sm_count();
  if (*blocks > most) *blocks = most;
  return cudaSuccess;
}

struct SortPlan {
  int64_t blocks, chunk;
  unsigned* counts;
  int* rows;
};
// Blocks that rank the places: each reads the counts of all, so not more than 65536 counts.
SortPlan plan_sort(Scratch& sc, const Dispatch& p) {
  const int64_t total = p.tokens * p.k, sms = ops_sm_count();
  SortPlan s;
  s.blocks = (total + kSortThreads - 1) / kSortThreads;
  if (s.blocks > sms) s.blocks = sms;
  const int64_t most = 65536 / (p.experts + 1);
  if (s.blocks > most) s.blocks = most < 8 ? 8 : most;
  s.chunk = (total + s.blocks - 1) / s.blocks;
  s.counts = sc.take<unsigned>(s.blocks * (p.experts + 1));
  s.rows = sc.take<int>(total);
  return s;
}

template <typename T, int VEC>
cudaError_t move(const Dispatch& p, Scratch& sc, cudaStream_t st) {
  MoveRows m{p.x, p.ldx, p.tokens, p.d, static_cast<int>(p.k), static_cast<int>(p.experts), p.idx, p.place, p.offsets, nullptr, p.xs};
  const int64_t total = p.tokens * p.k;
  if (total <= kFewPlaces)
    return launch_after(dispatch_few_kernel<T, VEC>, static_cast<unsigned>(p.tokens + 1), kThreads, sizeof(unsigned) * (p.experts + 1), st, m);
  const SortPlan s = plan_sort(sc, p);
  m.rows = s.rows;
  const size_t held = sizeof(unsigned) * static_cast<size_t>(p.experts + 1);
  cudaError_t e = launch_after(expert_count_kernel, static_cast<unsigned>(s.blocks), kSortThreads, held, st, p.idx, total, s.chunk, m.experts, s.counts);
  if (e == cudaSuccess)
    e = launch_after(expert_rank_kernel, static_cast<unsigned>(s.blocks), kSortThreads, (p.experts < kByWarp ? 2 + kSortWarps : 2) * held, st, p.idx, total, s.chunk, m.experts,
                     static_cast<const unsigned*>(s.counts), s.rows, p.place, p.offsets);
  if (e != cudaSuccess) return e;
  const int share = share_of(p.d, 16 / static_cast<int>(sizeof(T)));
  return launch_after(dispatch_kernel<T, VEC>, static_cast<unsigned>(blocks_of(p.tokens, share)), kThreads, 0, st, m, share);
}

JoinRows join_of(const Combine& p) {
  return JoinRows{p.ys, p.ldys, p.rows, p.tokens, p.d, static_cast<int>(p.k), p.place, p.weights, p.y, p.dy, p.lddy, nullptr, nullptr, nullptr, nullptr, p.dys, p.dweights};
}

template <typename T, int VEC>
cudaError_t backward(const Combine& p, Scratch& sc, cudaStream_t st) {
  JoinRows q = join_of(p);
  // (four pieces a thread: what a token costs beside them, its places and the sums over its threads, counts less.  With one piece
  // 120 us instead of 104 for 8192 x 8 rows of 2048 bf16 and 75 instead of 68 for 4093 x 6 of 2001; with eight 111 and 72.  With the
  // rows' blocks as they are now 100.6 and 65.)
  const int share = share_of(p.d, 4 * (VEC > 1 ? VEC : 4));
  int64_t token_blocks = blocks_of(p.tokens, share);
  const int64_t total = p.tokens * p.k;
  static PerDevice known;
  cudaError_t fits = blocks_at_once(combine_backward_kernel<T, VEC>, known, &token_blocks);
  if (fits != cudaSuccess) return fits;
  int64_t row_blocks = 0;
  if (p.rows == 0) q.dys = nullptr;
  if (q.dys) {
    q.listed = sc.take<unsigned>(p.rows);
    q.first = sc.take<int>(p.rows);
    q.last = sc.take<int>(p.rows);
    q.next = sc.take<int>(total);
    row_blocks = (p.rows + kRowsBlock - 1) / kRowsBlock;
    cudaError_t e = launch_after(clear_listed_kernel, static_cast<unsigned>((p.rows + kThreads - 1) / kThreads), kThreads, 0, st, q.listed, p.rows);
    const unsigned blocks = static_cast<unsigned>((total + kThreads - 1) / kThreads);
    if (e == cudaSuccess && blocks) e = launch_after(count_listed_kernel, blocks, kThreads, 0, st, p.place, total, q.listed, q.first, q.last, q.next, p.rows);
    if (e != cudaSuccess) return e;
  }
  if (token_blocks + row_blocks > INT32_MAX) return cudaErrorNotSupported;
  if (token_blocks + row_blocks == 0) return cudaSuccess;
  return launch_after(combine_backward_kernel<T, VEC>, static_cast<unsigned>(token_blocks + row_blocks), kThreads, 0, st, q, share, token_blocks);
}

}  // namespace

size_t dispatch_scratch_bytes(const Dispatch& p) {
  if (p.tokens * p.k <= kFewPlaces) return 0;
  Scratch sc;
  plan_sort(sc, p);
  return sc.used();
}

cudaError_t launch_dispatch(const Dispatch& p, Scratch& sc, cudaStream_t st) {
  if (p.tokens + 1 > INT32_MAX) return cudaErrorNotSupported;
  const bool f32 = p.dtype == kF32;
  const bool wide = whole_vectors(f32 ? 4 : 2, p.d, {p.x, p.xs}, {p.ldx});
  if (f32) return wide ? move<float, 4>(p, sc, st) : move<float, 1>(p, sc, st);
  return wide ? move<__nv_bfloat16, 8>(p, sc, st) : move<__nv_bfloat16, 1>(p, sc, st);
}

template <typename T, int VEC>
static cudaError_t forward(const Combine& p, cudaStream_t st) {
  // (two pieces a thread: 49 us instead of 51 for 8192 x 8 rows of 2048 bf16, 22 instead of 23.5 for 4093 x 6 of 1001 f32; dispatch, which
  // writes k rows for each it reads, takes 57 us with two and 53 with one)
  const int share = share_of(p.d, 2 * 16 / static_cast<int>(sizeof(T)));
  return launch_after(combine_kernel<T, VEC>, static_cast<unsigned>(blocks_of(p.tokens, share)), kThreads, 0, st, join_of(p), share);
}

cudaError_t launch_combine(const Combine& p, cudaStream_t st) {
  const bool f32 = p.dtype == kF32;
  const bool wide = whole_vectors(f32 ? 4 : 2, p.d, {p.ys, p.y}, {p.ldys});
  if (f32) return wide ? forward<float, 4>(p, st) : forward<float, 1>(p, st);
  return wide ? forward<__nv_bfloat16, 8>(p, st) : forward<__nv_bfloat16, 1>(p, st);
}

size_t combine_backward_scratch_bytes(const Combine& p) {
  Scratch sc;
  if (p.dys) {
    sc.take<unsigned>(p.rows);
    sc.take<int>(p.rows);
    sc.take<int>(p.rows);
    sc.take<int>(p.tokens * p.k);
  }
  return sc.used();
}

cudaError_t launch_combine_backward(const Combine& p, Scratch& sc, cudaStream_t st) {
  const bool f32 = p.dtype == kF32;
  const bool wide = whole_vectors(f32 ? 4 : 2, p.d, {p.dy, p.dweights ? p.ys : nullptr, p.dys}, {p.lddy, p.dweights ? p.ldys : 0});
  if (f32) return wide ? backward<float, 4>(p, sc, st) : backward<float, 1>(p, sc, st);
  return wide ? backward<__nv_bfloat16, 8>(p, sc, st) : backward<__nv_bfloat16, 1>(p, sc, st);
}

}  // namespace tk

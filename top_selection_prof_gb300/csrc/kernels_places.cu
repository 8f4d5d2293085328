// Products of a selection with a dictionary, and their gradients.
//
// A selection lists S places (r, c) with a value each, in order of value.  The
// two passes over it are sums by row (a reconstruction, or the gradient of an
// input) and sums by column (the gradient of a dictionary).  Flat positions
// are grouped first: each place takes a rank in its group by an atomic
// counter, groups take their bases from one running total, and the places are
// written to their slots.  Ranks and bases differ from run to run; the order
// in which a group is summed does not: its places are put in order of s where
// they are summed (a group of at most kPiece), or by a bitmap of s over the
// whole selection (a longer group, one block each).  A longer group is summed
// in pieces of kPiece places, and the piece that ends last adds the pieces up
// in their order.  So results do not depend on the order of the atomics.
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

constexpr int kPiece = 64;       // places summed by one warp or block at a time
constexpr int kBaseThreads = 256;
constexpr int kSortThreads = 512;
constexpr int64_t kBitmapBits = int64_t(1) << 20;  // places one bitmap of the sort covers (128 KB)
constexpr uint32_t kNoPlace = 0xffffffffu;

struct GroupHeader {
  unsigned total;   // places that lie in range
  unsigned pieces;  // pieces of long groups
  unsigned longs;   // long groups
};
struct PieceRec {
  unsigned group, index, slot0, count;  // piece `index` of a group whose first slot is slot0; the group's places
};
// Groups of one call, in its scratch.
struct Groups {
  GroupHeader* hdr;
  unsigned* count;    // per group
  unsigned* ticket;   // per piece slot: pieces of the group that are done (counted at its first slot)
  unsigned* start;    // per group
  uint32_t* rank;     // per place: its rank in its group as counted, or kNoPlace
  uint2* order;       // grouped places (s, other coordinate)
  uint2* sorted;      // long groups: the same in order of s
  PieceRec* pieces;
  unsigned* longs;    // long groups
  float* part;        // pieces x d sums
  float* part_bias;   // pieces sums of coefficients
  int64_t zero_bytes; // hdr, count and ticket lie together and start at zero
  int64_t n_groups, max_pieces, max_longs;
};

Groups plan_groups(Scratch& sc, int64_t total, int64_t groups, int64_t d, bool bias) {
  Groups g{};
  g.n_groups = groups;
  // a group in pieces has more than kPiece places, so at most 2 x places / kPiece pieces
  g.max_longs = total / (kPiece + 1);
  g.max_pieces = g.max_longs ? 2 * (total / kPiece) : 0;
  const size_t z0 = sc.used();
  g.hdr = sc.take<GroupHeader>(1);
  g.count = sc.take<unsigned>(groups);
  g.ticket = sc.take<unsigned>(g.max_pieces);
  g.zero_bytes = static_cast<int64_t>(sc.used() - z0);
  g.start = sc.take<unsigned>(groups);
  g.rank = sc.take<uint32_t>(total);
  g.order = sc.take<uint2>(total);
  g.sorted = sc.take<uint2>(g.max_longs ? total : 0);
  g.pieces = sc.take<PieceRec>(g.max_pieces);
  g.longs = sc.take<unsigned>(g.max_longs);
  g.part = sc.take<float>(g.max_pieces * d);
  g.part_bias = sc.take<float>(bias ? g.max_pieces : 0);
  return g;
}

// Row and column of place s; false when its position is out of range.
__device__ __forceinline__ bool locate(const Places& p, int64_t s, uint32_t* row, uint32_t* col) {
  const int64_t v = p.idx[s];
  if (p.per_row) {
    *row = static_cast<uint32_t>(s / p.count);
    *col = static_cast<uint32_t>(v);
    return v >= 0 && v < p.n;
  }
  if (v < 0) return false;
  const int64_t r = v / p.n;
  *row = static_cast<uint32_t>(r);
  *col = static_cast<uint32_t>(v - r * p.n);
  return r < p.rows;
}

template <typename T>
__device__ __forceinline__ float coef_of(const Coef& c, int64_t s) {
  if (!c.coef) return 0.0f;
  const float v = to_f32(static_cast<const T*>(c.coef)[s]);
  if (!c.gate) return v;
  return to_f32(static_cast<const T*>(c.gate)[s]) > 0.0f ? v : 0.0f;
}

// ---- grouping -----------------------------------------------------------------
template <bool BY_ROW, typename T>
__global__ void count_places_kernel(const Places p, const Groups g, T* dots) {
  const int64_t s = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (s >= p.total) return;
  uint32_t row, col;
  if (!locate(p, s, &row, &col)) {
    g.rank[s] = kNoPlace;
    if (dots) dots[s] = from_f32<T>(0.0f);
    return;
  }
  g.rank[s] = atomicAdd(&g.count[BY_ROW ? row : col], 1u);
}

// A base for every group, from a scan over the block's groups and one atomic
// on the running total; the pieces and the list of long groups likewise.
__global__ void __launch_bounds__(kBaseThreads) group_base_kernel(const Groups g) {
  __shared__ unsigned warp_sum[kBaseThreads / 32];
  __shared__ unsigned block_base;
  const int64_t i = int64_t(blockIdx.x) * kBaseThreads + threadIdx.x;
  const unsigned cnt = i < g.n_groups ? g.count[i] : 0u;
  unsigned incl = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(~0u, incl, o);
    if (static_cast<int>(threadIdx.x % 32) >= o) incl += t;
  }
  if (threadIdx.x % 32 == 31) warp_sum[threadIdx.x / 32] = incl;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned t = 0;
    for (int w = 0; w < kBaseThreads / 32; ++w) {
      const unsigned v = warp_sum[w];
      warp_sum[w] = t;
      t += v;
    }
    block_base = t ? atomicAdd(&g.hdr->total, t) : 0u;
  }
  __syncthreads();
  if (i >= g.n_groups) return;
  g.start[i] = block_base + warp_sum[threadIdx.x / 32] + incl - cnt;
  if (cnt > kPiece) {
    const unsigned np = (cnt + kPiece - 1) / kPiece;
    const unsigned slot0 = atomicAdd(&g.hdr->pieces, np);
    for (unsigned q = 0; q < np; ++q) g.pieces[slot0 + q] = PieceRec{static_cast<unsigned>(i), q, slot0, cnt};
    g.longs[atomicAdd(&g.hdr->longs, 1u)] = static_cast<unsigned>(i);
  }
}

template <bool BY_ROW>
__global__ void place_kernel(const Places p, const Groups g) {
  const int64_t s = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (s >= p.total) return;
  const uint32_t rank = g.rank[s];
  if (rank == kNoPlace) return;
  uint32_t row, col;
  locate(p, s, &row, &col);
  g.order[g.start[BY_ROW ? row : col] + rank] = make_uint2(static_cast<uint32_t>(s), BY_ROW ? col : row);
}

// Long groups in order of s: a bitmap of the places, kBitmapBits at a time;
// each set bit's rank is the number of bits before it.
template <bool BY_ROW>
__global__ void __launch_bounds__(kSortThreads) sort_long_kernel(const Places p, const Groups g, int64_t words) {
  extern __shared__ uint32_t bitmap[];
  __shared__ unsigned warp_sum[kSortThreads / 32];
  __shared__ unsigned window_total;
  for (unsigned l = blockIdx.x; l < g.hdr->longs; l += gridDim.x) {
    const unsigned group = g.longs[l];
    const unsigned cnt = g.count[group], start = g.start[group];
    unsigned done = 0;
    for (int64_t s0 = 0; s0 < p.total && done < cnt; s0 += words * 32) {
      for (int64_t i = threadIdx.x; i < words; i += kSortThreads) bitmap[i] = 0;
      __syncthreads();
      for (unsigned i = threadIdx.x; i < cnt; i += kSortThreads) {
        const int64_t at = int64_t(g.order[start + i].x) - s0;
        if (at >= 0 && at < words * 32) atomicOr(&bitmap[at >> 5], 1u << (at & 31));
      }
      __syncthreads();
      // each thread's words, in a run; the bits before it by a scan over the block
      const int64_t run = (words + kSortThreads - 1) / kSortThreads;
      const int64_t w0 = threadIdx.x * run, w1 = min(words, w0 + run);
      unsigned mine = 0;
      for (int64_t w = w0; w < w1; ++w) mine += __popc(bitmap[w]);
      unsigned incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned t = __shfl_up_sync(~0u, incl, o);
        if (static_cast<int>(threadIdx.x % 32) >= o) incl += t;
      }
      if (threadIdx.x % 32 == 31) warp_sum[threadIdx.x / 32] = incl;
      __syncthreads();
      if (threadIdx.x == 0) {
        unsigned t = 0;
        for (int w = 0; w < kSortThreads / 32; ++w) {
          const unsigned v = warp_sum[w];
          warp_sum[w] = t;
          t += v;
        }
        window_total = t;
      }
      __syncthreads();
      unsigned at = start + done + warp_sum[threadIdx.x / 32] + incl - mine;
      for (int64_t w = w0; w < w1; ++w) {
        for (uint32_t b = bitmap[w]; b; b &= b - 1) {
          const int64_t s = s0 + w * 32 + (__ffs(b) - 1);
          uint32_t row, col;
          locate(p, s, &row, &col);
          g.sorted[at++] = make_uint2(static_cast<uint32_t>(s), BY_ROW ? col : row);
        }
      }
      done += window_total;
      __syncthreads();
    }
  }
}

template <bool BY_ROW, typename T>
cudaError_t launch_grouping(const Places& p, const Groups& g, T* dots, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(g.hdr, 0, static_cast<size_t>(g.zero_bytes), st);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>((p.total + 255) / 256);
  if (!blocks) return cudaSuccess;  // every group is empty
  count_places_kernel<BY_ROW, T><<<blocks, 256, 0, st>>>(p, g, dots);
  group_base_kernel<<<static_cast<unsigned>((g.n_groups + kBaseThreads - 1) / kBaseThreads), kBaseThreads, 0, st>>>(g);
  place_kernel<BY_ROW><<<blocks, 256, 0, st>>>(p, g);
  if (g.max_longs) {
    const int64_t bits = p.total < kBitmapBits ? p.total : kBitmapBits;
    const int64_t words = (bits + 31) / 32;
    e = cudaFuncSetAttribute(sort_long_kernel<BY_ROW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kBitmapBits / 8));
    if (e != cudaSuccess) return e;
    const int64_t most = 4 * ops_sm_count();
    const unsigned grid = static_cast<unsigned>(g.max_longs < most ? g.max_longs : most);
    sort_long_kernel<BY_ROW><<<grid, kSortThreads, static_cast<size_t>(words) * 4, st>>>(p, g, words);
  }
  return cudaGetLastError();
}

// The places [first, first + cnt) of a group in order of s: entry i of out.
// `threads` threads of which this is `t`; the caller synchronises after it.
__device__ __forceinline__ void order_short(const uint2* src, int cnt, uint2* raw, int t, int threads) {
  for (int i = t; i < cnt; i += threads) raw[i] = src[i];
}
__device__ __forceinline__ int rank_short(const uint2* raw, int cnt, int i) {
  const uint32_t s = raw[i].x;
  int rank = 0;
  for (int j = 0; j < cnt; ++j) rank += raw[j].x < s;
  return rank;
}

struct Entry {
  uint32_t other;
  float coef;
};

// ---- sums by row ------------------------------------------------------------------
// A block takes one piece of a row: kRowTx threads across d (VEC values each),
// kRowTy places at a time, whose sums are added in shared memory in order.
constexpr int kRowTx = 64, kRowTy = 4, kRowThreads = kRowTx * kRowTy;

struct RowParams {
  RowSums r;
  Groups g;
  int64_t pieces_per_row;  // per_row selections: pieces of each row, in place
  int64_t d_tiles;
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kRowThreads) row_sums_kernel(const RowParams q) {
  __shared__ uint2 raw[kPiece];
  __shared__ Entry ent[kPiece];
  __shared__ float sums[kRowTy - 1][kRowTx * VEC];
  __shared__ bool last;
  const RowSums& r = q.r;
  const Places& p = r.places;
  const int64_t tile = blockIdx.x % q.d_tiles;
  int64_t w = blockIdx.x / q.d_tiles;
  const int t = threadIdx.x;
  // which piece
  int64_t row;
  unsigned n_pieces = 1, index = 0, slot0 = 0;
  int cnt;
  if (p.per_row) {
    row = w / q.pieces_per_row;
    index = static_cast<unsigned>(w % q.pieces_per_row);
    n_pieces = static_cast<unsigned>(q.pieces_per_row);
    slot0 = static_cast<unsigned>(row * q.pieces_per_row);
    const int64_t at = int64_t(index) * kPiece;
    cnt = static_cast<int>(min(int64_t(kPiece), p.count - at));
    if (t < cnt) {
      const int64_t s = row * p.count + at + t;
      const int64_t c = p.idx[s];
      const bool ok = c >= 0 && c < p.n;
      ent[t] = Entry{ok ? static_cast<uint32_t>(c) : kNoPlace, ok ? coef_of<T>(r.coef, s) : 0.0f};
    }
  } else if (w < q.g.max_pieces) {
    if (w >= q.g.hdr->pieces) return;
    const PieceRec rec = q.g.pieces[w];
    row = rec.group;
    index = rec.index;
    slot0 = rec.slot0;
    n_pieces = (rec.count + kPiece - 1) / kPiece;
    cnt = static_cast<int>(min(unsigned(kPiece), rec.count - index * kPiece));
    if (t < cnt) {
      const uint2 e = q.g.sorted[q.g.start[row] + index * kPiece + t];
      ent[t] = Entry{e.y, coef_of<T>(r.coef, e.x)};
    }
  } else {
    row = w - q.g.max_pieces;
    const unsigned c = q.g.count[row];
    if (c > kPiece) return;
    cnt = static_cast<int>(c);
    order_short(q.g.order + q.g.start[row], cnt, raw, t, kRowThreads);
    __syncthreads();
    if (t < cnt) ent[rank_short(raw, cnt, t)] = Entry{raw[t].y, coef_of<T>(r.coef, raw[t].x)};
  }
  __syncthreads();
  const int tx = t % kRowTx, ty = t / kRowTx;
  const int64_t j = tile * (kRowTx * VEC) + int64_t(tx) * VEC;
  const bool in = j < r.d;
  const T* wt = static_cast<const T*>(r.w) + j;
  float acc[VEC] = {};
  if (in) {
#pragma unroll 4
    for (int i = ty; i < cnt; i += kRowTy) {
      const Entry e = ent[i];
      if (e.other == kNoPlace) continue;
      Vec<T, VEC> v;
      v.load_nc(wt + int64_t(e.other) * r.ldw);
#pragma unroll
      for (int c = 0; c < VEC; ++c) acc[c] = fmaf(e.coef, v.v[c], acc[c]);
    }
  }
  if (ty > 0) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) sums[ty - 1][tx * VEC + c] = acc[c];
  }
  __syncthreads();
  if (ty == 0) {
#pragma unroll
    for (int o = 0; o < kRowTy - 1; ++o)
#pragma unroll
      for (int c = 0; c < VEC; ++c) acc[c] += sums[o][tx * VEC + c];
  }
  if (n_pieces > 1) {
    // this piece's sums, then the last piece of the row adds them all in order
    if (ty == 0 && in) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) q.g.part[int64_t(slot0 + index) * r.d + j + c] = acc[c];
      __threadfence();
    }
    __syncthreads();
    if (t == 0) last = atomicAdd(&q.g.ticket[int64_t(slot0) * q.d_tiles + tile], 1u) == n_pieces - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (ty == 0 && in) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) acc[c] = 0.0f;
#pragma unroll 4
      for (unsigned o = 0; o < n_pieces; ++o)
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[c] += __ldcg(&q.g.part[int64_t(slot0 + o) * r.d + j + c]);
    }
  }
  if (ty == 0 && in) {
    Vec<T, VEC> out;
    if (r.bias) {
      out.load_nc(static_cast<const T*>(r.bias) + j);
#pragma unroll
      for (int c = 0; c < VEC; ++c) out.v[c] += acc[c];
    } else {
#pragma unroll
      for (int c = 0; c < VEC; ++c) out.v[c] = acc[c];
    }
    out.store(static_cast<T*>(r.y) + row * r.d + j);
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T>
bool row_vectors(const RowSums& r) {
  constexpr int kVec = 16 / sizeof(T);
  return r.d % kVec == 0 && r.ldw % kVec == 0 && aligned16(r.w) && aligned16(r.y) && (!r.bias || aligned16(r.bias));
}

RowParams plan_rows(const RowSums& r, Scratch& sc) {
  RowParams q{};
  q.r = r;
  const int vec = (r.dtype == kF32 ? row_vectors<float>(r) : row_vectors<__nv_bfloat16>(r)) ? (r.dtype == kF32 ? 4 : 8) : 1;
  q.d_tiles = (r.d + kRowTx * vec - 1) / (kRowTx * vec);
  if (r.places.per_row) {
    q.pieces_per_row = r.places.count > kPiece ? (r.places.count + kPiece - 1) / kPiece : 1;
    if (q.pieces_per_row > 1) {
      q.g.ticket = sc.take<unsigned>(r.places.rows * q.pieces_per_row * q.d_tiles);
      q.g.part = sc.take<float>(r.places.rows * q.pieces_per_row * r.d);
    }
  } else {
    q.g = plan_groups(sc, r.places.total, r.places.rows, r.d, false);
    // one ticket a slot and tile of d
    q.g.ticket = sc.take<unsigned>(q.g.max_pieces * q.d_tiles);
  }
  return q;
}

template <typename T>
cudaError_t launch_rows_t(const RowParams& q, cudaStream_t st) {
  const RowSums& r = q.r;
  constexpr int kVec = 16 / sizeof(T);
  cudaError_t e = cudaSuccess;
  int64_t work;
  if (r.places.per_row) {
    work = r.places.rows * q.pieces_per_row;
    if (q.pieces_per_row > 1)
      e = cudaMemsetAsync(q.g.ticket, 0, sizeof(unsigned) * static_cast<size_t>(work * q.d_tiles), st);
  } else {
    work = q.g.max_pieces + r.places.rows;
    e = launch_grouping<true, T>(r.places, q.g, static_cast<T*>(nullptr), st);
    if (e == cudaSuccess && q.g.max_pieces)
      e = cudaMemsetAsync(q.g.ticket, 0, sizeof(unsigned) * static_cast<size_t>(q.g.max_pieces * q.d_tiles), st);
  }
  if (e != cudaSuccess) return e;
  work *= q.d_tiles;
  if (work > INT32_MAX) return cudaErrorInvalidValue;
  if (row_vectors<T>(r))
    row_sums_kernel<T, kVec><<<static_cast<unsigned>(work), kRowThreads, 0, st>>>(q);
  else
    row_sums_kernel<T, 1><<<static_cast<unsigned>(work), kRowThreads, 0, st>>>(q);
  return cudaGetLastError();
}

// ---- sums by column ---------------------------------------------------------------
// A warp takes one piece of a column and goes over d in tiles of 32 x VEC x
// kColChunks values: the column's row of w in registers, the rows of x of its
// places streamed past it, kColAhead places' loads in flight.
constexpr int kColWarps = 4, kColChunks = 2, kColAhead = 4;

struct ColParams {
  ColumnSums c;
  Groups g;
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kColWarps * 32) column_sums_kernel(const ColParams q) {
  __shared__ uint2 raw_all[kColWarps][kPiece];
  __shared__ Entry ent_all[kColWarps][kPiece];
  __shared__ uint32_t place_all[kColWarps][kPiece];
  __shared__ float dots_all[kColWarps][kPiece];
  const ColumnSums& c = q.c;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint2* raw = raw_all[warp];
  Entry* ent = ent_all[warp];
  uint32_t* place = place_all[warp];
  float* dots = dots_all[warp];
  const int64_t wk = int64_t(blockIdx.x) * kColWarps + warp;
  int64_t col;
  unsigned n_pieces = 1, index = 0, slot0 = 0;
  int cnt;
  if (wk < q.g.max_pieces) {
    if (wk >= q.g.hdr->pieces) return;
    const PieceRec rec = q.g.pieces[wk];
    col = rec.group;
    index = rec.index;
    slot0 = rec.slot0;
    n_pieces = (rec.count + kPiece - 1) / kPiece;
    cnt = static_cast<int>(min(unsigned(kPiece), rec.count - index * kPiece));
    for (int i = lane; i < cnt; i += 32) {
      const uint2 e = q.g.sorted[q.g.start[col] + index * kPiece + i];
      ent[i] = Entry{e.y, coef_of<T>(c.coef, e.x)};
      place[i] = e.x;
    }
  } else {
    col = wk - q.g.max_pieces;
    if (col >= q.g.n_groups) return;
    const unsigned n = q.g.count[col];
    if (n > kPiece) return;
    cnt = static_cast<int>(n);
    order_short(q.g.order + q.g.start[col], cnt, raw, lane, 32);
    __syncwarp();
    for (int i = lane; i < cnt; i += 32) {
      const int k = rank_short(raw, cnt, i);
      ent[k] = Entry{raw[i].y, coef_of<T>(c.coef, raw[i].x)};
      place[k] = raw[i].x;
    }
  }
  for (int i = lane; i < cnt; i += 32) dots[i] = 0.0f;
  __syncwarp();
  const T* x = static_cast<const T*>(c.x);
  const T* w = static_cast<const T*>(c.w);
  T* dw = static_cast<T*>(c.dw);
  const bool want_dots = c.dots != nullptr, want_dw = c.dw != nullptr;
  constexpr int kSpan = 32 * VEC * kColChunks;
  for (int64_t d0 = 0; d0 < c.d && (want_dots || want_dw); d0 += kSpan) {
    int64_t j[kColChunks];
    bool in[kColChunks];
    Vec<T, VEC> wv[kColChunks];
    float acc[kColChunks][VEC] = {};
#pragma unroll
    for (int e = 0; e < kColChunks; ++e) {
      j[e] = d0 + (e * 32 + lane) * VEC;
      in[e] = j[e] < c.d;
#pragma unroll
      for (int v = 0; v < VEC; ++v) wv[e].v[v] = 0.0f;
      if (want_dots && cnt && in[e]) wv[e].load_nc(w + col * c.ldw + j[e]);
    }
    for (int i0 = 0; i0 < cnt; i0 += kColAhead) {
      Vec<T, VEC> xv[kColAhead][kColChunks];
#pragma unroll
      for (int a = 0; a < kColAhead; ++a) {
        const bool have = i0 + a < cnt;
        const T* xr = x + int64_t(have ? ent[i0 + a].other : 0) * c.ldx;
#pragma unroll
        for (int e = 0; e < kColChunks; ++e) {
#pragma unroll
          for (int v = 0; v < VEC; ++v) xv[a][e].v[v] = 0.0f;
          if (have && in[e]) xv[a][e].load_nc(xr + j[e]);
        }
      }
#pragma unroll
      for (int a = 0; a < kColAhead; ++a) {
        if (i0 + a >= cnt) break;
        const float f = ent[i0 + a].coef;
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < kColChunks; ++e)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            acc[e][v] = fmaf(f, xv[a][e].v[v], acc[e][v]);
            dot = fmaf(xv[a][e].v[v], wv[e].v[v], dot);
          }
        if (want_dots) {
#pragma unroll
          for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
          if (lane == 0) dots[i0 + a] += dot;
        }
      }
    }
    if (want_dw) {
#pragma unroll
      for (int e = 0; e < kColChunks; ++e) {
        if (!in[e]) continue;
        if (n_pieces > 1) {
#pragma unroll
          for (int v = 0; v < VEC; ++v) q.g.part[int64_t(slot0 + index) * c.d + j[e] + v] = acc[e][v];
        } else {
          Vec<T, VEC> out;
#pragma unroll
          for (int v = 0; v < VEC; ++v) out.v[v] = acc[e][v];
          out.store(dw + col * c.d + j[e]);
        }
      }
    }
  }
  __syncwarp();
  if (want_dots)
    for (int i = lane; i < cnt; i += 32) static_cast<T*>(c.dots)[place[i]] = from_f32<T>(dots[i]);
  float sum = 0.0f;
  if (c.dbias) {
    for (int i = 0; i < cnt; ++i) sum += ent[i].coef;
    if (n_pieces == 1 && lane == 0) static_cast<T*>(c.dbias)[col] = from_f32<T>(sum);
  }
  if (n_pieces == 1) return;
  if (c.dbias && lane == 0) q.g.part_bias[slot0 + index] = sum;
  __threadfence();
  __syncwarp();
  unsigned seen = 0;
  if (lane == 0) seen = atomicAdd(&q.g.ticket[slot0], 1u);
  seen = __shfl_sync(~0u, seen, 0);
  if (seen != n_pieces - 1) return;
  __threadfence();
  if (want_dw) {
    for (int64_t j = int64_t(lane) * VEC; j < c.d; j += 32 * VEC) {
      Vec<T, VEC> out;
#pragma unroll
      for (int v = 0; v < VEC; ++v) out.v[v] = 0.0f;
#pragma unroll 4
      for (unsigned o = 0; o < n_pieces; ++o)
#pragma unroll
        for (int v = 0; v < VEC; ++v) out.v[v] += __ldcg(&q.g.part[int64_t(slot0 + o) * c.d + j + v]);
      out.store(dw + col * c.d + j);
    }
  }
  if (c.dbias && lane == 0) {
    float t = 0.0f;
    for (unsigned o = 0; o < n_pieces; ++o) t += __ldcg(&q.g.part_bias[slot0 + o]);
    static_cast<T*>(c.dbias)[col] = from_f32<T>(t);
  }
}

template <typename T>
cudaError_t launch_columns_t(const ColParams& q, cudaStream_t st) {
  const ColumnSums& c = q.c;
  constexpr int kVec = 16 / sizeof(T);
  cudaError_t e = launch_grouping<false, T>(c.places, q.g, static_cast<T*>(c.dots), st);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (q.g.max_pieces + q.g.n_groups + kColWarps - 1) / kColWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const bool vec = c.d % kVec == 0 && c.ldx % kVec == 0 && aligned16(c.x) && (!c.dots || (c.ldw % kVec == 0 && aligned16(c.w))) &&
                   (!c.dw || aligned16(c.dw));
  if (vec)
    column_sums_kernel<T, kVec><<<static_cast<unsigned>(blocks), kColWarps * 32, 0, st>>>(q);
  else
    column_sums_kernel<T, 1><<<static_cast<unsigned>(blocks), kColWarps * 32, 0, st>>>(q);
  return cudaGetLastError();
}

ColParams plan_columns(const ColumnSums& c, Scratch& sc) {
  ColParams q{};
  q.c = c;
  q.g = plan_groups(sc, c.places.total, c.places.n, c.dw ? c.d : 0, c.dbias != nullptr);
  return q;
}

}  // namespace

size_t row_sums_scratch_bytes(const RowSums& r) {
  Scratch sc;
  plan_rows(r, sc);
  return sc.used();
}
cudaError_t launch_row_sums(const RowSums& r, Scratch& sc, cudaStream_t st) {
  const RowParams q = plan_rows(r, sc);
  return r.dtype == kF32 ? launch_rows_t<float>(q, st) : launch_rows_t<__nv_bfloat16>(q, st);
}
size_t column_sums_scratch_bytes(const ColumnSums& c) {
  Scratch sc;
  plan_columns(c, sc);
  return sc.used();
}
cudaError_t launch_column_sums(const ColumnSums& c, Scratch& sc, cudaStream_t st) {
  const ColParams q = plan_columns(c, sc);
  return c.dtype == kF32 ? launch_columns_t<float>(q, st) : launch_columns_t<__nv_bfloat16>(q, st);
}

}  // namespace tk

// Products of a selection with a dictionary, and their gradients.
//
// A selection lists S places (r, c) with a value each, in order of value.  The
// two passes over it are sums by row (a reconstruction, or the gradient of an
// input) and sums by column (the gradient of a dictionary).  Flat positions
// are grouped first: each place takes a rank in its group by an atomic
// counter, groups take their bases from one running total, and the places are
// written to their slots.  Ranks and bases differ from run to run; the order
// in which a group is summed does not: a short group's places are put in
// order of s where they are summed, a long group's by a block of its own
// before that.  A long group is summed in pieces, whose sums are added eight at a
// time, level by level, by the warp of each eight that ends last (by a
// ticket).  So results do not depend on the order of the atomics, and nothing
// waits for another block.
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

// Places summed at a time (most; a group with more is long): by a warp or block of a row, by a warp of columns.
constexpr int kRowPiece = 64, kColPiece = 32;
constexpr int kThreads = 256, kSortThreads = 512;
constexpr int kSpan = 8;                       // groups next to each other that may share a task
constexpr int kGroupsBlock = 256;              // groups of one block of the base kernel: their places lie together
constexpr int kSortSmall = 512;               // places of a long group ordered by counting smaller ones
constexpr int64_t kBitmapBits = int64_t(1) << 18;  // places that one bitmap of a longer group covers (with its counts 64 KB)
constexpr uint32_t kNoPlace = 0xffffffffu;

struct GroupHeader {
  unsigned total;   // places that lie in range
  unsigned pieces;  // pieces of long groups
  unsigned longs;   // long groups
  unsigned tasks;   // warps' tasks of the sums by column
  unsigned taken;   // items taken by the warps that sum them, after each warp's first
};
// What one warp (or block) sums: a piece of a long group, or, by column, a few
// short groups next to each other.
struct __align__(16) Item {
  unsigned group, columns, start, places;  // first group and how many (0: a piece); where their places lie
  unsigned slot0, index, pieces, unused;   // piece `index` of a group in `pieces`, whose first slot is slot0
};
// A grouped place.
struct __align__(16) Entry {
  uint32_t s, other;  // the place and its other coordinate
  float coef;
  uint32_t group;
};
// Groups of one call, in its scratch.
struct Groups {
  GroupHeader* hdr;
  unsigned* count;    // per group
  unsigned* start;    // per group
  uint4* seen;        // per place: group, other coordinate, rank in the group as counted (kNoPlace: none), coefficient
  Entry* order;       // the places by group
  Entry* sorted;      // long groups in order of s
  Item* pieces;       // of long groups
  Item* tasks;        // sums by column (else null): short groups that share a warp
  unsigned* longs;
  unsigned* ticket;   // pieces of a long group (and tile of d) that are done, counted at its first slot; zero at first
  float* part;        // pieces x d sums, rows of part_ld
  float* part_bias;   // pieces sums of coefficients
  int64_t n_groups, max_pieces, max_longs, max_tasks, n_tickets;
  int64_t part_ld;
  int piece, share;   // most places of a piece, and of columns that share a warp
};

// The groupings that one call's kernels make together: by column, by row, or both.
struct Groupings {
  Groups g[2];
  bool by_row[2];
  int n;
};

Groups plan_groups(Scratch& sc, int64_t total, int64_t groups, int piece, int64_t d, int64_t d_tiles, bool bias, bool tasks) {
  Groups g{};
  g.n_groups = groups;
  g.piece = piece;
  g.share = piece < 16 ? piece : 16;
  // a long group has more than `piece` places, so at most 2 x places / piece pieces
  g.max_longs = total / (piece + 1);
  g.max_pieces = g.max_longs ? 2 * (total / piece) : 0;
  g.n_tickets = g.max_pieces * d_tiles;
  g.hdr = sc.take<GroupHeader>(1);
  g.count = sc.take<unsigned>(groups);
  g.start = sc.take<unsigned>(groups);
  g.seen = sc.take<uint4>(total);
  g.order = sc.take<Entry>(total);
  g.sorted = sc.take<Entry>(g.max_longs ? total : 0);
  g.pieces = sc.take<Item>(g.max_pieces);
  // a span of groups that is no one task has more than `share` places
  g.max_tasks = tasks ? (groups + kSpan - 1) / kSpan + (kSpan - 1) * (total / g.share) : 0;
  g.tasks = tasks ? sc.take<Item>(g.max_tasks) : nullptr;
  g.longs = sc.take<unsigned>(g.max_longs);
  g.ticket = sc.take<unsigned>(g.n_tickets);
  g.part_ld = (d + 3) / 4 * 4;
  g.part = sc.take<float>(g.max_pieces * g.part_ld);
  g.part_bias = sc.take<float>(bias ? g.max_pieces : 0);
  return g;
}

// Row and column of place s; false when its position is out of range.
__device__ __forceinline__ bool locate(const Places& p, int64_t s, uint32_t* row, uint32_t* col) {
  const int64_t v = p.idx[s];
  if (p.per_row) {
    *row = static_cast<uint32_t>(s) / static_cast<uint32_t>(p.count);
    *col = static_cast<uint32_t>(v);
    return v >= 0 && v < p.n;
  }
  if (v < 0) return false;
  if (v <= 0xffffffffll) {
    const uint32_t r = static_cast<uint32_t>(v) / static_cast<uint32_t>(p.n);
    *row = r;
    *col = static_cast<uint32_t>(v) - r * static_cast<uint32_t>(p.n);
    return r < p.rows;
  }
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
__global__ void __launch_bounds__(kThreads) zero_groups_kernel(const Groupings all) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  for (int k = 0; k < all.n; ++k) {
    const Groups& g = all.g[k];
    if (i == 0) *g.hdr = GroupHeader{0, 0, 0, 0, 0};
    if (i < g.n_groups) g.count[i] = 0;
    if (i < g.n_tickets) g.ticket[i] = 0;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) count_places_kernel(const Places p, const Coef c, const Groupings all, T* dots) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t s = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (s >= p.total) return;
  uint32_t row, col;
  const bool in = locate(p, s, &row, &col);
  const float coef = coef_of<T>(c, s);
  uint32_t rank[2] = {kNoPlace, kNoPlace};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < all.n && in) rank[k] = atomicAdd(&all.g[k].count[all.by_row[k] ? row : col], 1u);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < all.n)
      all.g[k].seen[s] = make_uint4(all.by_row[k] ? row : col, all.by_row[k] ? col : row, rank[k], __float_as_uint(coef));
  if (!in && dots) dots[s] = from_f32<T>(0.0f);
}

// Inclusive sum over the block's threads; *total: of all.  (Two barriers.)
template <int THREADS>
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned* total) {
  __shared__ unsigned warp_sum[THREADS / 32];
  unsigned incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(~0u, incl, o);
    if (static_cast<int>(threadIdx.x % 32) >= o) incl += t;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 31) warp_sum[threadIdx.x / 32] = incl;
  __syncthreads();
  unsigned before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const unsigned t = warp_sum[w];
    if (w < static_cast<int>(threadIdx.x / 32)) before += t;
    all += t;
  }
  *total = all;
  return before + incl;
}

// A base for every group, from a scan over the block's groups and one atomic
// on the running total; the pieces and the list of long groups likewise.
__global__ void __launch_bounds__(kGroupsBlock) group_base_kernel(const Groupings all) {
  __shared__ unsigned block_base, task_base;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t blocks0 = (all.g[0].n_groups + kGroupsBlock - 1) / kGroupsBlock;
  const int which = blockIdx.x >= blocks0;
  const Groups& g = all.g[which];
  const unsigned piece = g.piece, share = g.share;
  const int64_t i = (int64_t(blockIdx.x) - (which ? blocks0 : 0)) * kGroupsBlock + threadIdx.x;
  const unsigned cnt = i < g.n_groups ? g.count[i] : 0u;
  unsigned total;
  const unsigned incl = block_scan<kGroupsBlock>(cnt, &total);
  if (threadIdx.x == 0) block_base = total ? atomicAdd(&g.hdr->total, total) : 0u;
  __syncthreads();
  const unsigned start = block_base + incl - cnt;
  if (g.tasks) {
    // as many groups next to each other (8, 4 or 2, aligned) as hold at most g.share places, or one
    const int lane = threadIdx.x % 32;
    const unsigned s2 = cnt + __shfl_xor_sync(~0u, cnt, 1), s4 = s2 + __shfl_xor_sync(~0u, s2, 2);
    const unsigned s8 = s4 + __shfl_xor_sync(~0u, s4, 4);
    unsigned size = 1, places = cnt;
    if (s8 <= share) size = 8, places = s8;
    else if (s4 <= share) size = 4, places = s4;
    else if (s2 <= share) size = 2, places = s2;
    const bool leads = lane % size == 0 && places <= piece && i < g.n_groups;
    // (one atomic a block; with one a warp, all on one counter, 65536 groups took 6.8 us instead of 5.7)
    unsigned made;
    unsigned slot = block_scan<kGroupsBlock>(leads, &made) - leads;
    if (threadIdx.x == 0) task_base = made ? atomicAdd(&g.hdr->tasks, made) : 0u;
    __syncthreads();
    slot += task_base;
    if (leads)
      g.tasks[slot] = Item{static_cast<unsigned>(i), static_cast<unsigned>(min(int64_t(size), g.n_groups - i)), start, places,
                           0, 0, 1, 0};
  }
  if (i >= g.n_groups) return;
  g.start[i] = start;
  if (cnt > piece) {
    const unsigned np = (cnt + piece - 1) / piece;
    const unsigned slot0 = atomicAdd(&g.hdr->pieces, np);
    for (unsigned q = 0; q < np; ++q)
      g.pieces[slot0 + q] = Item{static_cast<unsigned>(i), 0, start + q * piece, min(piece, cnt - q * piece), slot0, q, np, 0};
    g.longs[atomicAdd(&g.hdr->longs, 1u)] = static_cast<unsigned>(i);
  }
}

__global__ void __launch_bounds__(kThreads) place_kernel(const Groupings all, int64_t total) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t s = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (s >= total) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k >= all.n) break;
    const Groups& g = all.g[k];
    const uint4 v = g.seen[s];
    if (v.z != kNoPlace) g.order[g.start[v.x] + v.z] = Entry{static_cast<uint32_t>(s), v.y, __uint_as_float(v.w), v.x};
  }
}

// Long groups in order of s, a block each: the rank of a place is the number
// of smaller s in its group, counted directly for up to kSortSmall places and
// by a bitmap of s, kBitmapBits at a time, beyond.
__global__ void __launch_bounds__(kSortThreads) sort_long_kernel(const Groupings all, int64_t total, int words) {
  extern __shared__ uint32_t sort_smem[];
  uint32_t* bitmap = sort_smem;
  uint32_t* before = sort_smem + words;  // set bits before each word
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned long0 = all.g[0].hdr->longs, n_long = long0 + (all.n > 1 ? all.g[1].hdr->longs : 0u);
  for (unsigned l = blockIdx.x; l < n_long; l += gridDim.x) {
    const Groups& g = all.g[l >= long0];
    const unsigned group = g.longs[l >= long0 ? l - long0 : l];
    const int cnt = static_cast<int>(g.count[group]);
    const Entry* src = g.order + g.start[group];
    Entry* dst = g.sorted + g.start[group];
    if (cnt <= kSortSmall) {
      constexpr int kEach = kSortSmall / kSortThreads;
      Entry e[kEach];
      int rank[kEach] = {};
      for (int i = threadIdx.x; i < (cnt + 3) / 4 * 4; i += kSortThreads) sort_smem[i] = i < cnt ? src[i].s : kNoPlace;
#pragma unroll
      for (int q = 0; q < kEach; ++q) {
        const int i = q * kSortThreads + threadIdx.x;
        if (i < cnt) e[q] = src[i];
        else e[q].s = 0;
      }
      __syncthreads();
      for (int j = 0; j < cnt; j += 4) {
        const uint4 t = *reinterpret_cast<const uint4*>(sort_smem + j);
#pragma unroll
        for (int q = 0; q < kEach; ++q)
          rank[q] += (t.x < e[q].s) + (t.y < e[q].s) + (t.z < e[q].s) + (t.w < e[q].s);
      }
#pragma unroll
      for (int q = 0; q < kEach; ++q)
        if (q * kSortThreads + static_cast<int>(threadIdx.x) < cnt) dst[rank[q]] = e[q];
      __syncthreads();
      continue;
    }
    unsigned done = 0;
    for (int64_t s0 = 0; s0 < total && done < static_cast<unsigned>(cnt); s0 += int64_t(words) * 32) {
      for (int i = threadIdx.x; i < words; i += kSortThreads) bitmap[i] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < cnt; i += kSortThreads) {
        const int64_t at = int64_t(src[i].s) - s0;
        if (at >= 0 && at < int64_t(words) * 32) atomicOr(&bitmap[at >> 5], 1u << (at & 31));
      }
      __syncthreads();
      // a thread's words in a run; the bits before it by a scan over the block
      const int run = (words + kSortThreads - 1) / kSortThreads;
      const int w0 = min(words, static_cast<int>(threadIdx.x) * run), w1 = min(words, w0 + run);
      unsigned bits = 0, held;
      for (int w = w0; w < w1; ++w) bits += __popc(bitmap[w]);
      unsigned at0 = block_scan<kSortThreads>(bits, &held) - bits;
      for (int w = w0; w < w1; ++w) {
        before[w] = at0;
        at0 += __popc(bitmap[w]);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < cnt; i += kSortThreads) {
        const Entry e = src[i];
        const int64_t at = int64_t(e.s) - s0;
        if (at >= 0 && at < int64_t(words) * 32)
          dst[done + before[at >> 5] + __popc(bitmap[at >> 5] & ((1u << (at & 31)) - 1u))] = e;
      }
      done += held;
      __syncthreads();
    }
  }
}

template <typename T>
cudaError_t launch_grouping(const Places& p, const Coef& c, const Groupings& all, T* dots, cudaStream_t st) {
  int64_t zero = 0, bases = 0, longs = 0;
  for (int k = 0; k < all.n; ++k) {
    const Groups& g = all.g[k];
    const int64_t z = g.n_groups > g.n_tickets ? g.n_groups : g.n_tickets;
    zero = z > zero ? z : zero;
    bases += (g.n_groups + kGroupsBlock - 1) / kGroupsBlock;
    longs += g.max_longs;
  }
  cudaError_t e = launch_after(zero_groups_kernel, static_cast<unsigned>((zero + kThreads - 1) / kThreads), kThreads, 0, st, all);
  const unsigned blocks = static_cast<unsigned>((p.total + kThreads - 1) / kThreads);
  if (e == cudaSuccess && blocks) e = launch_after(count_places_kernel<T>, blocks, kThreads, 0, st, p, c, all, dots);
  if (e != cudaSuccess) return e;
  e = launch_after(group_base_kernel, static_cast<unsigned>(bases), kGroupsBlock, 0, st, all);
  if (e != cudaSuccess || !blocks) return e;  // (no places: every group is empty)
  e = launch_after(place_kernel, blocks, kThreads, 0, st, all, p.total);
  if (e != cudaSuccess || !longs) return e;
  const int64_t bits = p.total < kBitmapBits ? p.total : kBitmapBits;
  int words = static_cast<int>((bits + 31) / 32);
  if (words < kSortSmall) words = kSortSmall;
  e = cudaFuncSetAttribute(sort_long_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kBitmapBits / 4));
  if (e != cudaSuccess) return e;
  const int64_t most = 3 * ops_sm_count();
  return launch_after(sort_long_kernel, static_cast<unsigned>(longs < most ? longs : most), kSortThreads,
                      static_cast<size_t>(words) * 8, st, all, p.total, words);
}

// ---- sums by row ------------------------------------------------------------------
constexpr int kRowAhead = 8;

// Adds up a long group's pieces, a warp at a time: called by the warp that has
// written piece `index` (of `pieces`, the first in slot `slot0`) to its slot,
// with values [j0, j1) of each slot's row of ld.  The warp that ends last of each eight
// adds them in their order into the first one's slot and goes on with the
// eights of the next level; the last of all writes dst = sum (+ bias).
constexpr unsigned kFan = 8;
struct Join {
  float* part;
  float* part_bias;   // nullable: a value a slot, added up the same way
  unsigned* ticket;   // of slot s and level l: [(s + l) * stride]; a level's eights lie eight slots apart or more
  int64_t stride, ld, j0, j1;
  unsigned slot0, index, pieces;
};
template <typename T>
__device__ __noinline__ void join_pieces(const Join& q, T* dst, const T* bias, T* dbias) {
  const int lane = threadIdx.x % 32;
  unsigned at = q.index, left = q.pieces, apart = 1;  // the sums of this level lie `apart` slots apart
  for (unsigned level = 0; left > 1; ++level) {
    const unsigned group = at / kFan, members = min(kFan, left - group * kFan);
    const unsigned slot = q.slot0 + group * kFan * apart;
    if (members > 1) {
      __threadfence();
      __syncwarp();
      unsigned seen = 0;
      if (lane == 0) seen = atomicAdd(&q.ticket[int64_t(slot + level) * q.stride], 1u);
      seen = __shfl_sync(~0u, seen, 0);
      if (seen != members - 1) return;
      __threadfence();
      const bool top = left <= kFan;
      // four values of each of the eight in flight (slots hold whole float4, j0 is one's first); more would cost the
      // kernels that call this their registers, and so their warps: with eight values 43 -> 76 us
      for (int64_t j = q.j0 + lane * 4; dst && j < q.j1; j += 128) {
        Vec<float, 4> t[kFan];
        float* src = q.part + int64_t(slot) * q.ld + j;
#pragma unroll
        for (unsigned m = 0; m < kFan; ++m)
          if (m < members) t[m].load_cg(src + int64_t(m) * apart * q.ld);
#pragma unroll
        for (unsigned m = 1; m < kFan; ++m)
          if (m < members) {
#pragma unroll
            for (int v = 0; v < 4; ++v) t[0].v[v] += t[m].v[v];
          }
        if (top) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (j + v < q.j1) dst[j + v] = from_f32<T>(t[0].v[v] + (bias ? to_f32(bias[j + v]) : 0.0f));
        } else {
          t[0].store(src);
        }
      }
      if (q.part_bias && lane == 0) {
        float sum = 0.0f;
        for (unsigned m = 0; m < members; ++m) sum += __ldcg(&q.part_bias[slot + m * apart]);
        if (top) *dbias = from_f32<T>(sum);
        else q.part_bias[slot] = sum;
      }
    }
    at = group;
    left = (left + kFan - 1) / kFan;
    apart *= kFan;
  }
}

struct RowParams {
  RowSums r;
  Groups g;
  int64_t pieces_per_row;  // per_row selections: pieces of each row, in place
  int64_t d_tiles;
};

// Many rows: a warp takes one piece of a row and one tile of 32 x VEC x CHUNKS
// values, places in order one after the other, AHEAD of them in flight.
constexpr int kRowWarps = 4, kRowChunks1 = 8;  // (chunks of rows that do not hold whole vectors)
template <typename T, int VEC, int CHUNKS, int AHEAD>
__global__ void __launch_bounds__(kRowWarps * 32) row_sums_warp_kernel(const RowParams q) {
  __shared__ Entry raw_all[kRowWarps][kRowPiece];
  __shared__ uint2 ent_all[kRowWarps][kRowPiece];  // other coordinate, coefficient
  grid_dependency_wait();
  grid_launch_dependents();
  const RowSums& r = q.r;
  const Places& p = r.places;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  Entry* raw = raw_all[warp];
  uint2* ent = ent_all[warp];
  const int64_t wk = int64_t(blockIdx.x) * kRowWarps + warp;
  const int64_t w = wk / q.d_tiles, tile = wk - w * q.d_tiles;
  int64_t row;
  unsigned n_pieces = 1, index = 0, slot0 = 0;
  int cnt = 0;
  if (p.per_row) {
    row = w / q.pieces_per_row;
    if (row >= p.rows) return;
    index = static_cast<unsigned>(w - row * q.pieces_per_row);
    n_pieces = static_cast<unsigned>(q.pieces_per_row);
    slot0 = static_cast<unsigned>(row * q.pieces_per_row);
    const int64_t at = int64_t(index) * kRowPiece;
    const int listed = static_cast<int>(min(int64_t(kRowPiece), p.count - at));
    for (int i0 = 0; i0 < listed; i0 += 32) {  // positions out of range are left out
      const int64_t s = row * p.count + at + i0 + lane;
      int64_t c = -1;
      float f = 0.0f;
      if (i0 + lane < listed) {
        c = p.idx[s];
        f = coef_of<T>(r.coef, s);
      }
      const bool held = c >= 0 && c < p.n;
      const unsigned who = __ballot_sync(~0u, held);
      if (held) ent[cnt + __popc(who & lanemask_lt())] = make_uint2(static_cast<uint32_t>(c), __float_as_uint(f));
      cnt += __popc(who);
    }
  } else if (w < p.rows) {
    row = w;
    const unsigned c = q.g.count[row];
    const unsigned start = q.g.start[row];
    if (c > kRowPiece) return;
    cnt = static_cast<int>(c);
    Entry e[2];
    int rank[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k * 32 + lane < cnt) raw[k * 32 + lane] = e[k] = q.g.order[start + k * 32 + lane];
    __syncwarp();
    for (int j = 0; j < cnt; ++j) {
      const uint32_t s = raw[j].s;
#pragma unroll
      for (int k = 0; k < 2; ++k) rank[k] += s < e[k].s;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k * 32 + lane < cnt) ent[rank[k]] = make_uint2(e[k].other, __float_as_uint(e[k].coef));
  } else {
    if (w - p.rows >= q.g.hdr->pieces) return;
    const Item rec = q.g.pieces[w - p.rows];
    row = rec.group;
    index = rec.index;
    slot0 = rec.slot0;
    n_pieces = rec.pieces;
    cnt = static_cast<int>(rec.places);
    for (int i = lane; i < cnt; i += 32) {
      const Entry e = q.g.sorted[rec.start + i];
      ent[i] = make_uint2(e.other, __float_as_uint(e.coef));
    }
  }
  __syncwarp();
  const int64_t j0 = tile * (32 * VEC * CHUNKS), j = j0 + int64_t(lane) * VEC;
  const T* wt = static_cast<const T*>(r.w) + j;
  bool in[CHUNKS];
  float acc[CHUNKS][VEC] = {};
#pragma unroll
  for (int h = 0; h < CHUNKS; ++h) in[h] = j + h * 32 * VEC < r.d;
#pragma unroll 1
  for (int i0 = 0; i0 < cnt; i0 += AHEAD) {
    Raw<T, VEC> v[AHEAD][CHUNKS];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
      if (i0 + a < cnt) {
        const T* row_w = wt + int64_t(ent[i0 + a].x) * r.ldw;
#pragma unroll
        for (int h = 0; h < CHUNKS; ++h)
          if (in[h]) v[a][h].load_nc(row_w + h * 32 * VEC);
      }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (i0 + a < cnt) {
        const float f = __uint_as_float(ent[i0 + a].y);
#pragma unroll
        for (int h = 0; h < CHUNKS; ++h)
          if (in[h]) {
            Vec<T, VEC> u;
            u.set_raw(v[a][h]);
#pragma unroll
            for (int c = 0; c < VEC; ++c) acc[h][c] = fmaf(f, u.v[c], acc[h][c]);
          }
      }
    }
  }
  T* y = static_cast<T*>(r.y) + row * r.d;
  const T* bias = static_cast<const T*>(r.bias);
  if (n_pieces > 1) {
#pragma unroll
    for (int h = 0; h < CHUNKS; ++h)
      if (in[h]) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) q.g.part[int64_t(slot0 + index) * q.g.part_ld + j + h * 32 * VEC + c] = acc[h][c];
      }
    const Join join{q.g.part, nullptr, q.g.ticket + tile, q.d_tiles, q.g.part_ld, j0, min(r.d, j0 + 32 * VEC * CHUNKS), slot0, index, n_pieces};
    join_pieces(join, y, bias, static_cast<T*>(nullptr));
    return;
  }
#pragma unroll
  for (int h = 0; h < CHUNKS; ++h)
    if (in[h]) {
      Vec<T, VEC> out;
#pragma unroll
      for (int c = 0; c < VEC; ++c) out.v[c] = 0.0f;
      if (bias) out.load_nc(bias + j + h * 32 * VEC);
#pragma unroll
      for (int c = 0; c < VEC; ++c) out.v[c] += acc[h][c];
      out.store(y + j + h * 32 * VEC);
    }
}

// Few rows: a block takes one piece of a row, kRowTx threads across d, the
// others different places, whose sums are added in shared memory in order.
constexpr int kRowTx = 16;
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) row_sums_kernel(const RowParams q) {
  constexpr int TX = kRowTx;
  constexpr int TY = kThreads / TX;
  __shared__ Entry raw[kRowPiece];
  __shared__ uint2 ent[kRowPiece];  // other coordinate, coefficient
  __shared__ float sums[TY - 1][TX * VEC];
  grid_dependency_wait();
  grid_launch_dependents();
  const RowSums& r = q.r;
  const Places& p = r.places;
  const int64_t tile = blockIdx.x % q.d_tiles;
  const int64_t w = blockIdx.x / q.d_tiles;
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
    const int64_t at = int64_t(index) * kRowPiece;
    cnt = static_cast<int>(min(int64_t(kRowPiece), p.count - at));
    if (t < cnt) {
      const int64_t s = row * p.count + at + t;
      const int64_t c = p.idx[s];
      ent[t] = make_uint2(c >= 0 && c < p.n ? static_cast<uint32_t>(c) : kNoPlace, __float_as_uint(coef_of<T>(r.coef, s)));
    }
  } else if (w < q.g.max_pieces) {
    if (w >= q.g.hdr->pieces) return;
    const Item rec = q.g.pieces[w];
    row = rec.group;
    index = rec.index;
    slot0 = rec.slot0;
    n_pieces = rec.pieces;
    cnt = static_cast<int>(rec.places);
    if (t < cnt) {
      const Entry e = q.g.sorted[rec.start + t];
      ent[t] = make_uint2(e.other, __float_as_uint(e.coef));
    }
  } else {
    row = w - q.g.max_pieces;
    const unsigned c = q.g.count[row];
    const unsigned start = q.g.start[row];
    if (c > kRowPiece) return;
    cnt = static_cast<int>(c);
    Entry e;
    if (t < cnt) raw[t] = e = q.g.order[start + t];
    __syncthreads();
    if (t < cnt) {
      int rank = 0;
      for (int j = 0; j < cnt; ++j) rank += raw[j].s < e.s;
      ent[rank] = make_uint2(e.other, __float_as_uint(e.coef));
    }
  }
  __syncthreads();
  const int tx = t % TX, ty = t / TX;
  const int64_t j = tile * (TX * VEC) + int64_t(tx) * VEC;
  const bool in = j < r.d;
  const T* wt = static_cast<const T*>(r.w) + j;
  float acc[VEC] = {};
  if (in) {
    for (int i0 = ty; i0 < cnt; i0 += TY * kRowAhead) {
      Raw<T, VEC> v[kRowAhead];
      float f[kRowAhead];
#pragma unroll
      for (int a = 0; a < kRowAhead; ++a) {
        f[a] = 0.0f;
        v[a].clear();
        const int i = i0 + a * TY;
        const uint2 e = i < cnt ? ent[i] : make_uint2(kNoPlace, 0u);
        if (e.x != kNoPlace) {
          v[a].load_nc(wt + int64_t(e.x) * r.ldw);
          f[a] = __uint_as_float(e.y);
        }
      }
#pragma unroll
      for (int a = 0; a < kRowAhead; ++a) {
        Vec<T, VEC> u;
        u.set_raw(v[a]);
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[c] = fmaf(f[a], u.v[c], acc[c]);
      }
    }
  }
  if (ty > 0) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) sums[ty - 1][tx * VEC + c] = acc[c];
  }
  __syncthreads();
  if (ty == 0) {
#pragma unroll
    for (int o = 0; o < TY - 1; ++o)
#pragma unroll
      for (int c = 0; c < VEC; ++c) acc[c] += sums[o][tx * VEC + c];
  }
  if (n_pieces > 1) {
    if (ty == 0 && in) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) q.g.part[int64_t(slot0 + index) * q.g.part_ld + j + c] = acc[c];
    }
    if (t >= 32) return;
    __syncwarp();
    const int64_t j0 = tile * (TX * VEC);
    const Join join{q.g.part, nullptr, q.g.ticket + tile, q.d_tiles, q.g.part_ld, j0, min(r.d, j0 + TX * VEC), slot0, index, n_pieces};
    join_pieces(join, static_cast<T*>(r.y) + row * r.d, static_cast<const T*>(r.bias), static_cast<T*>(nullptr));
    return;
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
int row_vec(const RowSums& r) {
  if (r.dtype == kF32) return row_vectors<float>(r) ? 4 : 1;
  return row_vectors<__nv_bfloat16>(r) ? 8 : 1;
}
// A warp a piece and tile when that gives every SM eight warps, else a block each (64 places of one row of 512 values:
// 12.6 us by one block's 64 threads across d, 4.8 us by four blocks' 16).
int64_t many_wide(const RowSums& r) { return row_vec(r) == 1 ? 32 * kRowChunks1 : 32 * row_vec(r); }
bool many_rows(const RowSums& r) {
  const int64_t wide = many_wide(r);
  return r.places.rows * ((r.d + wide - 1) / wide) >= 8 * ops_sm_count();
}

RowParams plan_rows(const RowSums& r, Scratch& sc) {
  RowParams q{};
  q.r = r;
  const int64_t wide = many_rows(r) ? many_wide(r) : int64_t(kRowTx) * row_vec(r);
  q.d_tiles = (r.d + wide - 1) / wide;
  if (r.places.per_row) {
    q.pieces_per_row = r.places.count > kRowPiece ? (r.places.count + kRowPiece - 1) / kRowPiece : 1;
    if (q.pieces_per_row > 1) {
      q.g.n_tickets = r.places.rows * q.pieces_per_row * q.d_tiles;
      q.g.hdr = sc.take<GroupHeader>(1);
      q.g.ticket = sc.take<unsigned>(q.g.n_tickets);
      q.g.part_ld = (r.d + 3) / 4 * 4;
      q.g.part = sc.take<float>(r.places.rows * q.pieces_per_row * q.g.part_ld);
    }
  } else {
    q.g = plan_groups(sc, r.places.total, r.places.rows, kRowPiece, r.d, q.d_tiles, false, false);
  }
  return q;
}

template <typename T, int VEC>
cudaError_t launch_rows_v(const RowParams& q, int64_t work, cudaStream_t st) {
  const bool many = many_rows(q.r);
  const int64_t grid = many ? (work + kRowWarps - 1) / kRowWarps : work;
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  if (many)
    return launch_after(row_sums_warp_kernel<T, VEC, VEC == 1 ? kRowChunks1 : 1, VEC == 1 ? 4 : 8>, static_cast<unsigned>(grid),
                        kRowWarps * 32, 0, st, q);
  return launch_after(row_sums_kernel<T, VEC>, static_cast<unsigned>(grid), kThreads, 0, st, q);
}

template <typename T>
cudaError_t launch_rows_t(const RowParams& q, cudaStream_t st) {
  const RowSums& r = q.r;
  constexpr int kVec = 16 / sizeof(T);
  const int64_t work = (r.places.per_row ? r.places.rows * q.pieces_per_row : q.g.max_pieces + r.places.rows) * q.d_tiles;
  return row_vectors<T>(r) ? launch_rows_v<T, kVec>(q, work, st) : launch_rows_v<T, 1>(q, work, st);
}

// ---- sums by column ---------------------------------------------------------------
// A warp takes items from a counter: pieces of long columns, or short columns
// next to each other, whose places (one a lane) it puts in order by column and
// s and streams through.  The places' rows of x (and, where a column begins,
// its row of w, for the dots) are copied to a ring of the warp's shared memory
// a tile of 32 x VEC x CHUNKS values at a time, kSlots - 1 places ahead, each
// lane the values that it will read itself; the sums stay in registers and are
// written where the column ends.  (131072 places of 512 bf16 values, with the
// dots: loads into registers two ahead leave a warp 0.7 us a place, 57 us in
// all; bulk copies of whole rows 95 us, one taking an SM some 70 ns.)
// FULL: every tile is whole.
constexpr int kColWarps = 4;

struct ColParams {
  ColumnSums c;
  Groups g;
};

template <typename T, int VEC, int CHUNKS, bool FULL, bool DOTS>
struct ColumnStream {
  static constexpr int kTile = 32 * VEC * CHUNKS;
  static constexpr int kTileBytes = kTile * sizeof(T);
  static constexpr int kSlots = DOTS ? 6 : 4;
  static constexpr int kSlotBytes = kTileBytes * (DOTS ? 2 : 1);
  static constexpr int kPairs = VEC / 2;
  const ColumnSums& c;
  unsigned char* ring;  // kSlots x kSlotBytes
  const Entry* ent;
  float* dots;
  float* part;  // where a piece's sums go (null: to dw)
  int lane, total, tiles;
  bool want_dw;
  Pair acc2[CHUNKS][kPairs ? kPairs : 1];  // sums, two a register pair
  float acc1[CHUNKS];                      // (VEC == 1)
  Pair wv2[DOTS ? CHUNKS : 1][kPairs ? kPairs : 1];  // the column's row of w
  float wv1[DOTS ? CHUNKS : 1];

  // The lane's first value of chunk h of a tile, in the row and in a slot.
  __device__ __forceinline__ int64_t at(int tile, int h) const { return int64_t(tile) * kTile + (h * 32 + lane) * VEC; }
  __device__ __forceinline__ int slot_at(int h) const { return (h * 32 + lane) * VEC * int(sizeof(T)); }
  __device__ __forceinline__ bool in(int tile, int h) const { return FULL || at(tile, h) < c.d; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int h = 0; h < CHUNKS; ++h) {
      acc1[h] = 0.0f;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) acc2[h][i] = Pair::of(0.0f, 0.0f);
    }
  }
  // The sums so far are a tile of column `col`.
  __device__ __forceinline__ void flush(int64_t col, int tile) {
#pragma unroll
    for (int h = 0; h < CHUNKS; ++h) {
      if (in(tile, h)) {
        Vec<T, VEC> out;
        if constexpr (VEC == 1) {
          out.v[0] = acc1[h];
        } else {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) acc2[h][i].get(&out.v[2 * i], &out.v[2 * i + 1]);
        }
        if (part) {
#pragma unroll
          for (int v = 0; v < VEC; ++v) part[at(tile, h) + v] = out.v[v];
        } else {
          out.store_stream(static_cast<T*>(c.dw) + col * c.d + at(tile, h));
        }
      }
    }
    clear();
  }
  // Place f (tile by tile) on its way to its slot; a group of copies in any case.
  __device__ __forceinline__ void issue(int f, int n) {
    if (f < n) {
      const int tile = tiles == 1 ? 0 : f / total, i = f - tile * total;
      const Entry e = ent[i];
      unsigned char* slot = ring + (f % kSlots) * kSlotBytes;
      const T* xr = static_cast<const T*>(c.x) + int64_t(e.other) * c.ldx;
#pragma unroll
      for (int h = 0; h < CHUNKS; ++h)
        if (in(tile, h)) copy_async<VEC>(reinterpret_cast<T*>(slot + slot_at(h)), xr + at(tile, h));
      if constexpr (DOTS) {
        if (i == 0 || ent[i - 1].group != e.group) {
          const T* wr = static_cast<const T*>(c.w) + int64_t(e.group) * c.ldw;
#pragma unroll
          for (int h = 0; h < CHUNKS; ++h)
            if (in(tile, h)) copy_async<VEC>(reinterpret_cast<T*>(slot + kTileBytes + slot_at(h)), wr + at(tile, h));
        }
      }
    }
    copy_async_commit();
  }
  __device__ __forceinline__ Raw<T, VEC> read(const unsigned char* slot, int tile, int h) const {
    Raw<T, VEC> r;
    r.clear();
    if (in(tile, h)) r.load(reinterpret_cast<const T*>(slot + slot_at(h)));
    return r;
  }
  __device__ __forceinline__ void run() {
    const int n = total * tiles;
    clear();
#pragma unroll
    for (int f = 0; f < kSlots - 1; ++f) issue(f, n);
    int i = 0, tile = 0;
    for (int f0 = 0; f0 < n; f0 += 4) {
      float dot[4] = {};
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        if (f0 + a < n) {
          issue(f0 + a + kSlots - 1, n);
          copy_async_wait_group<kSlots - 1>();
          const unsigned char* slot = ring + ((f0 + a) % kSlots) * kSlotBytes;
          const float coef = ent[i].coef;
          const uint32_t group = ent[i].group;
          const Pair f2 = Pair::of(coef, coef);
          if constexpr (DOTS) {
            if (i == 0 || ent[i - 1].group != group) {
#pragma unroll
              for (int h = 0; h < CHUNKS; ++h) {
                const Raw<T, VEC> r = read(slot + kTileBytes, tile, h);
                if constexpr (VEC == 1) {
                  wv1[h] = to_f32(r.u);
                } else {
#pragma unroll
                  for (int k = 0; k < kPairs; ++k) wv2[h][k] = r.pair(k);
                }
              }
            }
          }
          Pair dot2 = Pair::of(0.0f, 0.0f);
#pragma unroll
          for (int h = 0; h < CHUNKS; ++h) {
            const Raw<T, VEC> xv = read(slot, tile, h);
            if constexpr (VEC == 1) {
              const float t = to_f32(xv.u);
              acc1[h] = fmaf(coef, t, acc1[h]);
              if constexpr (DOTS) dot[a] = fmaf(t, wv1[h], dot[a]);
            } else {
#pragma unroll
              for (int k = 0; k < kPairs; ++k) {
                const Pair t = xv.pair(k);
                acc2[h][k].fma(f2, t);
                if constexpr (DOTS) dot2.fma(t, wv2[h][k]);
              }
            }
          }
          if constexpr (DOTS && VEC > 1) {
            float lo, hi;
            dot2.get(&lo, &hi);
            dot[a] = lo + hi;
          }
          if (ent[i + 1].group != group) {  // (past the last place: no group's number)
            if (want_dw) flush(group, tile);
            else clear();
          }
          if (++i == total) {
            i = 0;
            ++tile;
          }
        }
      }
      if constexpr (DOTS) {
        // four sums over the lanes, by exchanging halves until a lane holds one
#pragma unroll
        for (int h = 2, o = 16; h >= 1; h /= 2, o /= 2) {
#pragma unroll
          for (int k = 0; k < h; ++k) {
            const bool high = lane & o;
            const float give = high ? dot[k] : dot[k + h];
            dot[k] = (high ? dot[k + h] : dot[k]) + __shfl_xor_sync(~0u, give, o);
          }
        }
#pragma unroll
        for (int o = 4; o; o /= 2) dot[0] += __shfl_xor_sync(~0u, dot[0], o);
        if (tiles == 1) {
          if (lane % 8 == 0 && f0 + lane / 8 < n) dots[f0 + lane / 8] = dot[0];
        } else {
          // one after the other: in a short list two of the four may be tiles of one place
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            if (lane == 8 * a && f0 + a < n) {
              const int t = (f0 + a) / total, k = f0 + a - t * total;
              dots[k] = (t ? dots[k] : 0.0f) + dot[0];
            }
            __syncwarp();
          }
        }
      }
    }
  }
  // Zeros to a row of dw.
  __device__ __forceinline__ void zeros(int64_t col) const {
    Vec<T, VEC> out;
#pragma unroll
    for (int v = 0; v < VEC; ++v) out.v[v] = 0.0f;
    for (int64_t j = lane * VEC; j < c.d; j += 32 * VEC) out.store_stream(static_cast<T*>(c.dw) + col * c.d + j);
  }
};

template <typename T, int VEC, int CHUNKS, bool FULL, bool DOTS>
__global__ void __launch_bounds__(kColWarps * 32, DOTS ? 4 : 6) column_sums_kernel(const ColParams q) {
  extern __shared__ __align__(16) unsigned char rings[];
  __shared__ Entry ent_all[kColWarps][kColPiece + 1];
  __shared__ Entry raw_all[kColWarps][kColPiece];  // the next item's places on their way
  __shared__ Item item_all[kColWarps][2];          // and the records of the two next items
  __shared__ float dots_all[kColWarps][kColPiece];
  static_assert(kColPiece == 32, "a place a lane");
  grid_dependency_wait();
  grid_launch_dependents();
  const ColumnSums& c = q.c;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  Entry* ent = ent_all[warp];
  Entry* raw = raw_all[warp];
  Item* items = item_all[warp];
  float* dots = dots_all[warp];
  T* dw = static_cast<T*>(c.dw);
  T* dbias = static_cast<T*>(c.dbias);
  using Stream = ColumnStream<T, VEC, CHUNKS, FULL, DOTS>;
  Stream st{c, rings + warp * (Stream::kSlots * Stream::kSlotBytes), ent, dots, nullptr, lane, 0,
            static_cast<int>((c.d + Stream::kTile - 1) / Stream::kTile), dw != nullptr};
  const unsigned pieces = q.g.hdr->pieces, work = pieces + q.g.hdr->tasks, step = gridDim.x * kColWarps;
  // Records and places are copied to shared memory ahead of their use: the record two items ahead, the places one.
  auto fetch_item = [&](unsigned wk, int slot) {
    if (wk < work && lane < 2) {
      const Item* from = wk < pieces ? q.g.pieces + wk : q.g.tasks + (wk - pieces);
      copy_async16(reinterpret_cast<uint4*>(items + slot) + lane, reinterpret_cast<const uint4*>(from) + lane);
    }
  };
  auto fetch_places = [&](unsigned wk, int slot) {
    if (wk < work && lane < static_cast<int>(items[slot].places))
      copy_async16(raw + lane, (items[slot].columns ? q.g.order : q.g.sorted) + items[slot].start + lane);
  };
  // Each warp's first two items are its own; the others it takes from a counter, three ahead.
  unsigned wk = blockIdx.x * kColWarps + warp, next = wk + step, after = 0;
  // (what the counter gives is not touched before it is needed, an item later)
  fetch_item(wk, 0);
  fetch_item(next, 1);
  if (lane == 0) after = atomicAdd(&q.g.hdr->taken, 1u);
  copy_async_wait();
  __syncwarp();
  fetch_places(wk, 0);
  for (unsigned turn = 0; wk < work; turn ^= 1) {
    copy_async_wait();
    __syncwarp();
    const Item item = items[turn];
    const int64_t c0 = item.group;
    const int total = static_cast<int>(item.places);
    const unsigned n_pieces = item.pieces, slot = item.slot0 + item.index;
    Entry e{kNoPlace, 0, 0.0f, kNoPlace};
    if (lane < total) e = raw[lane];
    __syncwarp();
    wk = next;
    next = 2 * step + __shfl_sync(~0u, after, 0);
    fetch_item(next, turn);
    fetch_places(wk, turn ^ 1);
    if (lane == 0) after = atomicAdd(&q.g.hdr->taken, 1u);
    int rank = lane;
    unsigned empty = 0;  // columns of the item without a place
    if (item.columns) {
      empty = ~__reduce_or_sync(~0u, lane < total ? 1u << (e.group - item.group) : 0u) & ((1u << item.columns) - 1u);
      if (total > 1) {
        // groups (their place in the item, 3 bits) above s (29 bits): one number to compare
        const uint32_t key = ((e.group - item.group) << 29) | e.s;
        rank = 0;
#pragma unroll 4
        for (int i = 0; i < total; ++i) rank += __shfl_sync(~0u, key, i) < key;
      }
    }
    if (lane < total) ent[rank] = e;
    if (lane == 0) ent[total].group = kNoPlace;
    __syncwarp();
    st.total = total;
    st.part = n_pieces > 1 ? q.g.part + int64_t(slot) * q.g.part_ld : nullptr;
    if (dw || DOTS) st.run();
    if (dw)
      for (unsigned b = empty; b; b &= b - 1) st.zeros(c0 + __ffs(b) - 1);
    __syncwarp();
    if (DOTS && lane < total) static_cast<T*>(c.dots)[ent[lane].s] = from_f32<T>(dots[lane]);
    float sum = 0.0f;
    if (dbias) {
      for (unsigned b = empty; b; b &= b - 1)
        if (lane == 0) dbias[c0 + __ffs(b) - 1] = from_f32<T>(0.0f);
      for (int i = 0; i < total; ++i) {
        sum += ent[i].coef;
        if (n_pieces == 1 && ent[i + 1].group != ent[i].group) {
          if (lane == 0) dbias[ent[i].group] = from_f32<T>(sum);
          sum = 0.0f;
        }
      }
    }
    if (n_pieces == 1) continue;
    if (dbias && lane == 0) q.g.part_bias[slot] = sum;
    const Join join{q.g.part, dbias ? q.g.part_bias : nullptr, q.g.ticket, 1, q.g.part_ld, 0, c.d, item.slot0, item.index, n_pieces};
    join_pieces(join, dw ? dw + c0 * c.d : nullptr, static_cast<const T*>(nullptr), dbias ? dbias + c0 : nullptr);
  }
}

template <typename T, int VEC, int CHUNKS, bool FULL, bool DOTS>
cudaError_t launch_columns_d(const ColParams& q, cudaStream_t st) {
  using Stream = ColumnStream<T, VEC, CHUNKS, FULL, DOTS>;
  auto kernel = column_sums_kernel<T, VEC, CHUNKS, FULL, DOTS>;
  constexpr int kSmem = kColWarps * Stream::kSlots * Stream::kSlotBytes;
  static PerDevice fits;  // blocks that fit an SM (the attribute, too, is the device's)
  std::atomic<int>* known = fits.here();
  int each = known ? known->load() : 0;
  if (!each) {
    int n = 0;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kColWarps * 32, kSmem);
    if (e != cudaSuccess) return e;
    each = n < 1 ? 1 : n;
    if (known) *known = each;
  }
  const int64_t blocks = (q.g.max_pieces + q.g.max_tasks + kColWarps - 1) / kColWarps, fit = int64_t(each) * ops_sm_count();
  return launch_after(kernel, static_cast<unsigned>(blocks < fit ? blocks : fit), kColWarps * 32, kSmem, st, q);
}
template <typename T, int VEC, int CHUNKS, bool FULL>
cudaError_t launch_columns_v(const ColParams& q, cudaStream_t st) {
  return q.c.dots ? launch_columns_d<T, VEC, CHUNKS, FULL, true>(q, st)
                  : launch_columns_d<T, VEC, CHUNKS, FULL, false>(q, st);
}

bool column_vectors(const ColumnSums& c) {
  const int vec = c.dtype == kF32 ? 4 : 8;
  return c.d % vec == 0 && c.ldx % vec == 0 && aligned16(c.x) && (!c.dots || (c.ldw % vec == 0 && aligned16(c.w))) &&
         (!c.dw || aligned16(c.dw));
}

template <typename T>
cudaError_t launch_columns_t(const ColParams& q, cudaStream_t st) {
  const ColumnSums& c = q.c;
  constexpr int kVec = 16 / sizeof(T);
  if (!column_vectors(c)) return launch_columns_v<T, 1, 8, false>(q, st);
  return c.d % (64 * kVec) == 0 ? launch_columns_v<T, kVec, 2, true>(q, st) : launch_columns_v<T, kVec, 2, false>(q, st);
}

ColParams plan_columns(const ColumnSums& c, Scratch& sc) {
  ColParams q{};
  q.c = c;
  // Pieces small enough for three to each of 16 warps an SM: where a few columns hold most places, one of 32 places of 771
  // f32 values kept its warp for 67 us.
  int piece = kColPiece;
  while (piece > 8 && c.places.total < int64_t(3) * piece * 16 * ops_sm_count()) piece /= 2;
  q.g = plan_groups(sc, c.places.total, c.places.n, piece, c.dw ? c.d : 0, 1, c.dbias != nullptr, true);
  return q;
}

}  // namespace

size_t sums_scratch_bytes(const ColumnSums* c, const RowSums* r) {
  Scratch sc;
  if (c) plan_columns(*c, sc);
  if (r) plan_rows(*r, sc);
  return sc.used();
}

cudaError_t launch_sums(const ColumnSums* c, const RowSums* r, Scratch& sc, cudaStream_t st) {
  ColParams cols{};
  RowParams rows{};
  Groupings all{};
  if (c) {
    cols = plan_columns(*c, sc);
    all.g[all.n++] = cols.g;
  }
  if (r) {
    rows = plan_rows(*r, sc);
    if (!r->places.per_row) {
      all.by_row[all.n] = true;
      all.g[all.n++] = rows.g;
    } else if (rows.pieces_per_row > 1) {  // (only its tickets, at zero)
      Groupings one{};
      one.g[0] = rows.g;
      one.n = 1;
      const cudaError_t e = launch_after(zero_groups_kernel, static_cast<unsigned>((rows.g.n_tickets + kThreads - 1) / kThreads),
                                         kThreads, 0, st, one);
      if (e != cudaSuccess) return e;
    }
  }
  const Places& p = c ? c->places : r->places;
  const Coef& coef = c ? c->coef : r->coef;
  const bool f32 = (c ? c->dtype : r->dtype) == kF32;
  cudaError_t e = cudaSuccess;
  if (all.n)
    e = f32 ? launch_grouping<float>(p, coef, all, static_cast<float*>(c ? c->dots : nullptr), st)
            : launch_grouping<__nv_bfloat16>(p, coef, all, static_cast<__nv_bfloat16*>(c ? c->dots : nullptr), st);
  if (e == cudaSuccess && c) e = f32 ? launch_columns_t<float>(cols, st) : launch_columns_t<__nv_bfloat16>(cols, st);
  if (e == cudaSuccess && r) e = f32 ? launch_rows_t<float>(rows, st) : launch_rows_t<__nv_bfloat16>(rows, st);
  return e;
}

}  // namespace tk

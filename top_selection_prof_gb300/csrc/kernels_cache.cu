// The positions of a key-value cache that stay, by accumulated attention weight.
//
// A head's score is the sum of the attention weights that its queries gave a
// position, held in f32.  What a call adds is summed in pairs of f32: the error
// of each addition is kept in the second, which is brought below the first's
// last bit again after every few rows.  (Without that it grew with the rows, and
// what was rounded off it too: 2^14 weights of 2^-26 beside a one were off by two
// half steps, 2^16 by eight.)  With u = 2^-24, K rows at a time and S the sum of the magnitudes,
// a row's addition to the second, at most (1 + K) u S, rounds off u of that: (K + 3) / 2 u^2 S
// a row on average, 5.5 u^2 S at most here, and joining the groups of a block 8 u^2 S each.  So a
// score is off by half a step and at most (rows + 32) 2^-45 S, and only where scores lie
// that close can a choice depend on how a sum was split.
//
// evict: sums by position over all SMs; the choice, a cluster a head: the score of
// the last one kept by two or three digits of its key, then the kept positions in
// order by counting; and the rows of both caches moved to their new places.
// replace: one token, one launch: a cluster a head adds the weights, finds the
// least score and writes the new row over it.
//
// One GB300, inputs changing between calls: 8 heads x 32768 positions x 128 queries bf16,
// 4096 kept of 128 + 128 values (102 MB): 36 us, of which the sums take 17 (67 MB), the
// choice 11 (eight barriers of a cluster and the scans between them), the rows 6 (34 MB); 48 heads x 5001 f32, up to 1021
// rows of 72 + 72 kept: 27 us, of which the rows 9 (56 MB).  Replacing one of 4096 slots in 512 heads, four bf16 weights a
// slot (51 MB): 16.7 us, and 13.3 where three inputs in turn are still in the L2 in part; in 8 heads of 2048: 4.8 us
// in a graph, launch and barriers.  (Blocks of 256 threads, four an SM, so that 512 heads run at once: with 512, two an SM,
// 19 us instead of 16.5.)
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostBlocks = 8;   // of a cluster

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// hi + lo.  A value that is not finite ends up in hi alone.
struct Sum2 {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float s = hi + v, b = s - hi;
    lo += (hi - (s - b)) + (v - b);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum2& o) {
    add(o.hi);
    lo += o.lo;
  }
  // lo to below hi's last bit, after a few additions.
  __device__ __forceinline__ void settle() {
    const float s = hi + lo;
    if (!(fabsf(s) < INFINITY)) return;
    lo -= s - hi;
    hi = s;
  }
  __device__ __forceinline__ float value() const { return fabsf(hi) < INFINITY ? hi + lo : hi; }
};
// A weight that is NaN (of a query whose mask left nothing) counts as 0.
__device__ __forceinline__ float counted(float w) { return w == w ? w : 0.0f; }

__device__ __forceinline__ int64_t clamped(int64_t v, int64_t most) { return v < 0 ? 0 : v > most ? most : v; }

// ---- sums by position ------------------------------------------------------------
struct WeightSums {
  View weights;       // batch, query head, query
  int64_t group, queries, capacity;
  unsigned heads, chunks;  // (32-bit: a 64-bit division takes a hundred instructions, in every thread)
  View score;         // batch, head
  const int64_t* lengths;
  float* out;         // batch x heads x capacity
};
constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32, kFewLanes = 8;

// Two sums of two f32 each, side by side.
struct Sum2Pair {
  Pair hi = Pair::of(0.0f, 0.0f), lo = Pair::of(0.0f, 0.0f);
  __device__ __forceinline__ static Pair plus(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
  }
  __device__ __forceinline__ static Pair minus(Pair a, Pair b) {
    Pair r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
  }
  __device__ __forceinline__ void add(Pair v) {
    const Pair s = plus(hi, v), b = minus(s, hi);
    lo = plus(lo, plus(minus(hi, minus(s, b)), minus(v, b)));
    hi = s;
  }
  // (an infinity may become NaN, and its sum is made anew)
  __device__ __forceinline__ void settle() {
    const Pair s = plus(hi, lo);
    lo = minus(lo, minus(s, hi));
    hi = s;
  }
};

// What one of LANES threads holds of LANES x VEC (or LANES x 4) positions: 16 bytes side by side, or four values LANES apart.
template <typename T, int VEC, int LANES>
struct Places {
  static constexpr int kWide = VEC > 1 ? VEC : 4;
  Raw<T, VEC> r[VEC > 1 ? 1 : kWide];
  __device__ __forceinline__ static int at(int lane, int e) { return VEC > 1 ? lane * VEC + e : e * LANES + lane; }
  // (positions behind `left`, which no sum is taken of, are read at the row's start; the last vector of a row may reach past its
  // length, not past the capacity)
  __device__ __forceinline__ static void offsets(int* off, int lane, int64_t left) {
#pragma unroll
    for (int e = 0; e < (VEC > 1 ? 1 : kWide); ++e) off[e] = at(lane, e) < left ? at(lane, e) : 0;
  }
  __device__ __forceinline__ void load(const T* row, const int* off) {
#pragma unroll
    for (int e = 0; e < (VEC > 1 ? 1 : kWide); ++e) r[e].load_nc(row + off[e]);
  }
  __device__ __forceinline__ Pair pair(int i) const {
    if constexpr (VEC > 1) return r[0].pair(i);
    else return Pair::of(to_f32(r[2 * i].u), to_f32(r[2 * i + 1].u));
  }
};

// A block: LANES pieces of positions of one head, the head's query rows dealt to its groups of LANES threads (a warp; eight where there
// are few positions: 294 heads x 80 positions x 480 queries bf16 42 -> 25 us for evict), kAhead of them under way.  (Four blocks an SM with eight rows
// each under way: two with sixteen took 41.5 us instead of 38.5 for evict as a whole, six with four 42.)
template <typename T, int VEC, int kAhead, int LANES = 32>
__global__ void __launch_bounds__(kSumThreads, 4) weight_sums_kernel(const WeightSums p) {
  using P = Places<T, VEC, LANES>;
  constexpr int kWide = P::kWide, kGroups = kSumThreads / LANES;
  __shared__ float2 part[kGroups][LANES * kWide];
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned bh = blockIdx.x / p.chunks, b = bh / p.heads, h = bh % p.heads;
  const int64_t len = clamped(p.lengths[b], p.capacity), at0 = int64_t(blockIdx.x - bh * p.chunks) * LANES * kWide;
  if (at0 >= len) return;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  Sum2Pair sum[kWide / 2];
  const int n = static_cast<int>(p.group * p.queries), queries = static_cast<int>(p.queries);
  const T* base = static_cast<const T*>(p.weights.data) + b * p.weights.batch + h * p.group * p.weights.head + at0;
  static_assert(LANES * kWide <= kSumThreads, "a position a thread at the end");
  const bool sums = threadIdx.x < LANES * kWide && at0 + threadIdx.x < len;
  const float before = sums ? static_cast<const float*>(p.score.data)[b * p.score.batch + h * p.score.head + at0 + threadIdx.x] : 0.0f;
  int off[VEC > 1 ? 1 : kWide];
  P::offsets(off, lane, len - at0);
  // (a group's rows are mostly as far apart as a head's own)
  const bool even = p.weights.head == p.queries * p.weights.row;
  const int64_t step = kGroups * p.weights.row;
  const T* row = base + group * p.weights.row;
  for (int i0 = group; i0 < n; i0 += kGroups * kAhead) {
    P v[kAhead];
    const bool all = i0 + (kAhead - 1) * kGroups < n;
#pragma unroll
    for (int a = 0; a < kAhead; ++a, row += step) {
      const int i = i0 + a * kGroups;
      if (!all && i >= n) break;
      if (!even) row = base + i / queries * p.weights.head + i % queries * p.weights.row;
      v[a].load(row, off);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (!all && i0 + a * kGroups >= n) break;
#pragma unroll
      for (int e = 0; e < kWide / 2; ++e) sum[e].add(v[a].pair(e));
    }
    if (i0 + kGroups * kAhead < n) {  // (the last ones' are joined, and settled, by the block)
#pragma unroll
      for (int e = 0; e < kWide / 2; ++e) sum[e].settle();
    }
  }
#pragma unroll
  for (int e = 0; e < kWide / 2; ++e) {
    float h0, h1, l0, l1;
    sum[e].hi.get(&h0, &h1);
    sum[e].lo.get(&l0, &l1);
    part[group][P::at(lane, 2 * e)] = make_float2(h0, l0);
    part[group][P::at(lane, 2 * e + 1)] = make_float2(h1, l1);
  }
  __syncthreads();
  if (!sums) return;
  const int at = threadIdx.x;
  Sum2 all;
  all.add(before);
  bool number = true;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    number = number && part[g][at].x == part[g][at].x;
    all.add(Sum2{part[g][at].x, part[g][at].y});
    all.settle();
  }
  if (!number) {  // a weight is NaN or infinite: anew, without the NaN ones
    all = Sum2{};
    all.add(before);
    for (int q = 0; q < n; ++q) {
      all.add(counted(to_f32(base[(q / queries) * p.weights.head + (q % queries) * p.weights.row + at])));
      all.settle();
    }
  }
  p.out[int64_t(bh) * p.capacity + at0 + at] = all.value();
}

// ---- the choice -------------------------------------------------------------------
struct Choice {
  const float* score;     // batch x heads rows, `ld` apart by head and `ld_batch` by batch
  int64_t ld_batch, ld, capacity;
  unsigned heads;
  const int64_t* lengths;
  int64_t keep, recent;
  float* out_score;       // batch x heads x keep
  int64_t* kept;
  int64_t* out_lengths;
};
constexpr int kDigits = 2048;  // 11 bits of a key at a time (the last 10)

struct __align__(16) ChoiceShared {
  unsigned hist[kDigits];      // this block's; zero between digits
  unsigned total[kDigits];     // the cluster's
  unsigned warp_sum[kWarps];
  unsigned found, above, held;
  unsigned over[kMostBlocks], even[kMostBlocks];  // of each block, in every block
};

// Sum over the threads before this one; *all: of the block.
__device__ __forceinline__ unsigned scan_before(ChoiceShared& s, unsigned v, unsigned* all) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  unsigned incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s.warp_sum[warp] = incl;
  __syncthreads();
  unsigned before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const unsigned t = s.warp_sum[w];
    if (w < warp) before += t;
    sum += t;
  }
  *all = sum;
  __syncthreads();
  return before + incl - v;
}

// Up to EACH positions a thread, in a run, whose keys stay in registers; 0: as many as it takes, read anew in each pass.
template <int EACH>
__global__ void __launch_bounds__(kThreads, 2) choice_kernel(const Choice p) {
  __shared__ ChoiceShared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
  for (int i = threadIdx.x; i < kDigits; i += kThreads) s.hist[i] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned bh = blockIdx.x / static_cast<unsigned>(blocks), b = bh / p.heads, h = bh % p.heads;
  const float* score = p.score + b * p.ld_batch + h * p.ld;
  const int64_t len = clamped(p.lengths[b], p.capacity);
  const int64_t kept = min(len, p.keep), old = len - min(p.recent, len);  // the last ones stay
  const unsigned want = static_cast<unsigned>(len > p.keep ? p.keep - (len - old) : old);  // of the others
  // this thread's run of positions
  const int64_t each = (len + blocks * kThreads - 1) / kThreads >> (31 - __clz(blocks));  // (blocks: a power of two)
  const int64_t begin = min(len, (int64_t(rank) * kThreads + threadIdx.x) * each), end = min(len, begin + each);
  const bool choose = want < old;
  // (in 32 bits, by the number in the run: how many there are, and how many of them are not recent)
  const int mine = static_cast<int>(end - begin), mine_old = static_cast<int>(clamped(old - begin, mine));
  float held[EACH ? EACH : 1];
  if constexpr (EACH > 0) {
#pragma unroll
    for (int e = 0; e < EACH; ++e) held[e] = e < mine ? score[begin + e] : 0.0f;
  }
  auto score_at = [&](int e) -> float {
    if constexpr (EACH > 0) return held[e];
    else return score[begin + e];
  };
  auto key_at = [&](int e) -> uint32_t { return order_key_f32(__float_as_uint(score_at(e))); };
  auto run = [&](int n, auto f) {
    if constexpr (EACH > 0) {
#pragma unroll
      for (int e = 0; e < EACH; ++e)
        if (e < n) f(e);
    } else {
      for (int e = 0; e < n; ++e) f(e);
    }
  };
  cluster_sync();               // (every block has started before another reaches into its memory)
  uint32_t key = 0, mask = 0;   // of the last one kept
  unsigned left = want;         // of those with the key's bits under the mask
  if (choose && want > 0) {
#pragma unroll 1
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit == 2 ? 10 : 11;
      run(mine_old, [&](int e) {
        const uint32_t k = key_at(e);
        if ((k & mask) == key) atomicAdd(&s.hist[(~k >> shift) & ((1u << bits) - 1)], 1u);
      });
      cluster_sync();
      const int share = kDigits / blocks;
      for (int i = rank * share + threadIdx.x; i < (rank + 1) * share; i += kThreads) {
        unsigned n = 0;
        for (int q = 0; q < blocks; ++q) n += cluster.map_shared_rank(&s, q)->hist[i];
        for (int q = 0; q < blocks; ++q) cluster.map_shared_rank(&s, q)->total[i] = n;
      }
      cluster_sync();
      unsigned n[kDigits / kThreads], sum = 0, all;
      const uint4 four = *reinterpret_cast<const uint4*>(&s.total[threadIdx.x * 4]);
      n[0] = four.x, n[1] = four.y, n[2] = four.z, n[3] = four.w;
      *reinterpret_cast<uint4*>(&s.hist[threadIdx.x * 4]) = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < kDigits / kThreads; ++q) sum += n[q];
      unsigned before = scan_before(s, sum, &all);
#pragma unroll
      for (int q = 0; q < kDigits / kThreads; ++q) {
        if (before < left && left <= before + n[q]) {
          s.found = threadIdx.x * (kDigits / kThreads) + q;
          s.above = before;
          s.held = n[q];
        }
        before += n[q];
      }
      __syncthreads();
      key |= (~s.found & ((1u << bits) - 1)) << shift;
      mask |= ((1u << bits) - 1) << shift;
      left -= s.above;
      const bool all_of_them = s.held == left;
      __syncthreads();
      if (all_of_them) break;  // (the digits below do not matter)
    }
  }
  // kept: the recent ones, scores above the key's, and the first `left` of those that equal it
  auto state = [&](int e) -> int {  // 2: kept, 1: equal, 0
    if (e >= mine_old || !choose) return 2;
    if (want == 0) return 0;
    const uint32_t k = key_at(e) & mask;
    return k > key ? 2 : k == key ? 1 : 0;
  };
  unsigned over = 0, even = 0, all_over, all_even;
  run(mine, [&](int e) {
    const int st = state(e);
    over += st == 2;
    even += st == 1;
  });
  if constexpr (EACH > 0) {  // both sums in one: less than 2^16 each
    static_assert(EACH * kThreads < 65536, "halves of 32 bits");
    unsigned all;
    const unsigned both = scan_before(s, over << 16 | even, &all);
    over = both >> 16, even = both & 0xffff, all_over = all >> 16, all_even = all & 0xffff;
  } else {
    over = scan_before(s, over, &all_over);
    even = scan_before(s, even, &all_even);
  }
  if (threadIdx.x < blocks) {
    ChoiceShared* peer = cluster.map_shared_rank(&s, threadIdx.x);
    peer->over[rank] = all_over;
    peer->even[rank] = all_even;
  }
  cluster_sync();
  for (int q = 0; q < rank; ++q) {
    over += s.over[q];
    even += s.even[q];
  }
  int64_t slot = int64_t(bh) * p.keep + over + min(even, left);
  run(mine, [&](int e) {
    const int st = state(e);
    const bool stays = st == 2 || (st == 1 && even < left);
    even += st == 1;
    if (!stays) return;
    p.kept[slot] = begin + e;
    p.out_score[slot] = score_at(e);
    ++slot;
  });
  for (int64_t i = kept + rank * kThreads + threadIdx.x; i < p.keep; i += int64_t(blocks) * kThreads) {
    p.kept[int64_t(bh) * p.keep + i] = -1;
    p.out_score[int64_t(bh) * p.keep + i] = 0.0f;
  }
  if (h == 0 && rank == 0 && threadIdx.x == 0) p.out_lengths[b] = kept;
}

// ---- moving rows ------------------------------------------------------------------
struct MoveKept {
  View in[2];          // keys, values
  void* out[2];        // batch x heads x keep x dim
  int dim[2];
  const int64_t* kept;
  int64_t keep;
  unsigned heads, chunks;  // runs of rows in a head
  int used, rows;      // threads a row, and rows that a block has threads for
};
constexpr int kMoveThreads = 256;
// A block: p.rows rows of a head times kMoveTogether, whose loads are under way together.
template <typename T, int VEC>
__global__ void __launch_bounds__(kMoveThreads) move_kept_kernel(const MoveKept p) {
  constexpr int kTogether = VEC > 1 ? 2 : 1, kEach = VEC > 1 ? 1 : 4;
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned bh = blockIdx.x / p.chunks, b = bh / p.heads, h = bh % p.heads;
  const int mine = threadIdx.x / p.used, at = threadIdx.x % p.used;
  if (mine >= p.rows) return;
  const int64_t i0 = int64_t(blockIdx.x - bh * p.chunks) * (p.rows * kTogether) + mine;
  const int64_t* kept = p.kept + int64_t(bh) * p.keep;
  int64_t from[kTogether];
#pragma unroll
  for (int r = 0; r < kTogether; ++r) from[r] = i0 + r * p.rows < p.keep ? kept[i0 + r * p.rows] : -1;
  const int most = max(p.dim[0], p.dim[1]);
  const T* src[2];
  T* dst[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    src[w] = static_cast<const T*>(p.in[w].data) + b * p.in[w].batch + h * p.in[w].head;
    dst[w] = static_cast<T*>(p.out[w]) + (int64_t(bh) * p.keep + i0) * p.dim[w];
  }
  // (the loads of both first, and without vectors four values of each)
  for (int c0 = at * VEC; c0 < most; c0 += p.used * VEC * kEach) {
    Raw<T, VEC> v[kTogether][2][kEach];
#pragma unroll
    for (int r = 0; r < kTogether; ++r)
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int c = c0 + e * p.used;
          v[r][w][e].clear();
          if (from[r] >= 0 && c < p.dim[w]) v[r][w][e].load_nc(src[w] + from[r] * p.in[w].row + c);
        }
#pragma unroll
    for (int r = 0; r < kTogether; ++r) {
      if (i0 + r * p.rows >= p.keep) break;
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int c = c0 + e * p.used;
          T* to = dst[w] + r * p.rows * p.dim[w] + c;
          if (c >= p.dim[w]) continue;
          if constexpr (VEC == 1) *to = v[r][w][e].u;
          else __stcs(reinterpret_cast<uint4*>(to), v[r][w][e].u);
        }
    }
  }
}

// ---- one token ----------------------------------------------------------------------
// A cluster a head: adds the group's weights to the scores, finds the slot and writes the token there.  A thread holds WIDE slots
// side by side, whose weights, score and positions are all under way at once; where rows are not on 16-byte boundaries, four that
// lie a block's width apart.
constexpr int kReplaceThreads = 256, kReplaceWarps = kReplaceThreads / 32;
template <typename W, int WIDE>
__global__ void __launch_bounds__(kReplaceThreads, 4) replace_kernel(const Replace p) {
  __shared__ uint64_t warp_least[kReplaceWarps];
  __shared__ uint64_t leasts[kMostBlocks];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned bh = blockIdx.x / static_cast<unsigned>(blocks), heads = static_cast<unsigned>(p.heads), b = bh / heads, h = bh % heads;
  const int64_t seen = max(p.lengths[b], int64_t(0)), len = min(seen, p.capacity);
  float* score = static_cast<float*>(p.score.data) + b * p.score.batch + h * p.score.head;
  int64_t* positions = static_cast<int64_t*>(p.positions.data) + b * p.positions.batch + h * p.positions.head;
  const W* weights = static_cast<const W*>(p.weights.data);
  if (weights) weights += b * p.weights.batch + h * p.group * p.weights.head;
  const int n = weights ? static_cast<int>(p.group * p.queries) : 0, queries = static_cast<int>(p.queries);
  const bool even = p.weights.head == p.queries * p.weights.row;  // (a group's rows as far apart as a head's own)
  const bool full = seen >= p.capacity;
  uint64_t least = ~uint64_t(0);  // (score, slot) of the least that may go
  constexpr int kHeld = WIDE > 1 ? WIDE : 4;
  auto slot_of = [](int64_t i, int e) { return WIDE > 1 ? i + e : i + e * kReplaceThreads; };
  for (int64_t i = int64_t(rank) * kReplaceThreads * kHeld + threadIdx.x * WIDE; i < len; i += int64_t(blocks) * kReplaceThreads * kHeld) {
    // (a run's slots behind `len` are read, not written: they lie within the capacity)
    Sum2 sum[kHeld];
    unsigned may = 0;  // slots that may go
    if constexpr (WIDE > 1) {
#pragma unroll
      for (int e = 0; e < WIDE; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(score + i + e);
        sum[e].hi = v.x, sum[e + 1].hi = v.y, sum[e + 2].hi = v.z, sum[e + 3].hi = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kHeld; ++e) sum[e].hi = slot_of(i, e) < len ? score[slot_of(i, e)] : 0.0f;
    }
    if (full) {  // (with recent == 0 too: a slot's position may lie behind the length, of a token that was taken back)
      if constexpr (WIDE > 1) {
#pragma unroll
        for (int e = 0; e < WIDE; e += 2) {
          const longlong2 v = *reinterpret_cast<const longlong2*>(positions + i + e);
          may |= (v.x < seen - p.recent ? 1u << e : 0) | (v.y < seen - p.recent ? 2u << e : 0);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kHeld; ++e) may |= slot_of(i, e) < len && positions[slot_of(i, e)] < seen - p.recent ? 1u << e : 0;
      }
    }
    constexpr int kAhead = 4, kParts = WIDE > 1 ? 1 : kHeld;
    for (int r0 = 0; r0 < n; r0 += kAhead) {
      Raw<W, WIDE> v[kAhead][kParts];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int r = r0 + a, g = even ? 0 : r / queries;
        const W* row = weights + g * p.weights.head + (r - g * queries) * p.weights.row;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          v[a][q].clear();
          if (r < n && slot_of(i, q) < len) v[a][q].load_nc(row + slot_of(i, q));
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          Vec<W, WIDE> x;
          x.set_raw(v[a][q]);
#pragma unroll
          for (int e = 0; e < WIDE; ++e) sum[q + e].add(counted(x.v[e]));
        }
      }
      if (r0 + kAhead < n) {
#pragma unroll
        for (int e = 0; e < kHeld; ++e) sum[e].settle();
      }
    }
    float value[kHeld];
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      value[e] = sum[e].value();
      if (may >> e & 1)
        least = min(least, static_cast<uint64_t>(order_key_f32(__float_as_uint(value[e]))) << 32 | static_cast<uint32_t>(slot_of(i, e)));
    }
    if (n) {
      if (WIDE > 1 && i + WIDE <= len) {
        if constexpr (WIDE > 1) {
#pragma unroll
          for (int e = 0; e < WIDE; e += 4) *reinterpret_cast<float4*>(score + i + e) = make_float4(value[e], value[e + 1], value[e + 2], value[e + 3]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kHeld; ++e)
          if (slot_of(i, e) < len) score[slot_of(i, e)] = value[e];
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(~0u, least, o));
  if (threadIdx.x % 32 == 0) warp_least[threadIdx.x / 32] = least;
  cluster_sync();
  if (threadIdx.x < blocks) {
    for (int w = 0; w < kReplaceWarps; ++w) least = min(least, warp_least[w]);
    *cluster.map_shared_rank(&leasts[rank], threadIdx.x) = least;
  }
  cluster_sync();
  for (int q = 0; q < blocks; ++q) least = q ? min(least, leasts[q]) : leasts[0];
  // (where every slot is recent, the token is not stored)
  const int64_t slot = seen < p.capacity ? seen : least == ~uint64_t(0) ? -1 : static_cast<int64_t>(static_cast<uint32_t>(least));
  if (rank != 0) return;
  if (threadIdx.x == 0) {
    p.slots[bh] = slot;
    if (slot >= 0) {
      score[slot] = 0.0f;
      positions[slot] = seen;
    }
  }
  if (slot < 0) return;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const View& in = w ? p.value : p.key;
    const View& out = w ? p.values : p.keys;
    const int64_t dim = w ? p.value_dim : p.key_dim;
    const int64_t src = b * in.batch + h * in.head, dst = b * out.batch + h * out.head + slot * out.row;
    for (int64_t c = threadIdx.x; c < dim; c += kReplaceThreads) {
      if (p.dtype == kF32) static_cast<float*>(out.data)[dst + c] = static_cast<const float*>(in.data)[src + c];
      else static_cast<__nv_bfloat16*>(out.data)[dst + c] = static_cast<const __nv_bfloat16*>(in.data)[src + c];
    }
  }
}

// Blocks of a cluster a head: more where heads are few, `on_sm` on each SM, down to `least` positions each.
int blocks_for(int64_t rows, int64_t positions, int64_t least, int on_sm) {
  int blocks = 1;
  while (blocks < kMostBlocks && rows * blocks * 2 <= on_sm * ops_sm_count() && positions > blocks * least) blocks *= 2;
  return blocks;
}

template <typename P>
cudaError_t launch_clusters(void (*kernel)(P), const P& p, int64_t rows, int blocks, int threads, cudaStream_t st) {
  if (rows * blocks > INT32_MAX) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

bool aligned_view(const View& v, int64_t size) {
  return (reinterpret_cast<uintptr_t>(v.data) | static_cast<uintptr_t>(v.batch * size) | static_cast<uintptr_t>(v.head * size) |
          static_cast<uintptr_t>(v.row * size)) % 16 == 0;
}

template <typename T>
cudaError_t add_weights(const Evict& p, float* out, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  const bool wide = aligned_view(p.weights, sizeof(T)) && p.capacity % kVec == 0;
  const int held = wide ? kVec : 4;
  const bool few = p.capacity <= 16 * held;  // (a warp's threads would mostly have none)
  const int64_t each = (few ? kFewLanes : 32) * held;
  const int64_t chunks = (p.capacity + each - 1) / each, blocks = chunks * p.batch * p.heads;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  const WeightSums w{p.weights, p.group, p.queries, p.capacity, static_cast<unsigned>(p.heads), static_cast<unsigned>(chunks), p.score, p.lengths, out};
  const unsigned grid = static_cast<unsigned>(blocks);
  if (few)
    return wide ? launch_after(weight_sums_kernel<T, kVec, 4, kFewLanes>, grid, kSumThreads, 0, st, w)
                : launch_after(weight_sums_kernel<T, 1, 4, kFewLanes>, grid, kSumThreads, 0, st, w);
  // (few rows a warp: four at a time and more blocks an SM)
  if (p.group * p.queries <= 4 * kSumWarps || !wide)
    return wide ? launch_after(weight_sums_kernel<T, kVec, 4>, grid, kSumThreads, 0, st, w) : launch_after(weight_sums_kernel<T, 1, 4>, grid, kSumThreads, 0, st, w);
  return launch_after(weight_sums_kernel<T, kVec, 8>, grid, kSumThreads, 0, st, w);
}

template <typename T>
cudaError_t move_kept(const Evict& p, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  const int64_t size = sizeof(T);
  const bool wide = aligned_view(p.keys, size) && aligned_view(p.values, size) && p.key_dim % kVec == 0 && p.value_dim % kVec == 0 &&
                    (reinterpret_cast<uintptr_t>(p.out_keys) | reinterpret_cast<uintptr_t>(p.out_values)) % 16 == 0;
  const int dim = static_cast<int>(p.key_dim > p.value_dim ? p.key_dim : p.value_dim);
  // whole rows by as many threads as they have pieces (18 of 16 bytes: 14 rows a block, not 8), or longer ones in turns
  const int pieces = (dim + (wide ? kVec : 4) - 1) / (wide ? kVec : 4), used = pieces < kMoveThreads ? pieces : kMoveThreads, rows = kMoveThreads / used;
  const int64_t each = rows * (wide ? 2 : 1), chunks = (p.keep + each - 1) / each, blocks = chunks * p.batch * p.heads;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  const MoveKept m{{p.keys, p.values}, {p.out_keys, p.out_values}, {static_cast<int>(p.key_dim), static_cast<int>(p.value_dim)}, p.out_kept, p.keep,
                   static_cast<unsigned>(p.heads), static_cast<unsigned>(chunks), used, rows};
  return wide ? launch_after(move_kept_kernel<T, kVec>, static_cast<unsigned>(blocks), kMoveThreads, 0, st, m)
              : launch_after(move_kept_kernel<T, 1>, static_cast<unsigned>(blocks), kMoveThreads, 0, st, m);
}

}  // namespace

size_t evict_scratch_bytes(const Evict& p) {
  Scratch sc;
  if (p.weights.data) sc.take<float>(p.batch * p.heads * p.capacity);
  return sc.used();
}

cudaError_t launch_evict(const Evict& p, Scratch& sc, cudaStream_t st) {
  Choice c{static_cast<const float*>(p.score.data), p.score.batch, p.score.head, p.capacity, static_cast<unsigned>(p.heads), p.lengths, p.keep,
           p.recent, p.out_score, p.out_kept, p.out_lengths};
  if (p.weights.data) {
    float* sums = sc.take<float>(p.batch * p.heads * p.capacity);
    const cudaError_t e = p.weights_dtype == kF32 ? add_weights<float>(p, sums, st) : add_weights<__nv_bfloat16>(p, sums, st);
    if (e != cudaSuccess) return e;
    c.score = sums;
    c.ld_batch = p.heads * p.capacity;
    c.ld = p.capacity;
  }
  const int64_t rows = p.batch * p.heads;
  const int blocks = blocks_for(rows, p.capacity, 2048, 2);
  // positions a thread: in registers up to 16
  const int64_t each = (p.capacity + int64_t(blocks) * kThreads - 1) / (int64_t(blocks) * kThreads);
  cudaError_t e = launch_clusters(each <= 4 ? choice_kernel<4> : each <= 8 ? choice_kernel<8> : each <= 16 ? choice_kernel<16> : choice_kernel<0>, c, rows, blocks, kThreads, st);
  if (e != cudaSuccess) return e;
  return p.dtype == kF32 ? move_kept<float>(p, st) : move_kept<__nv_bfloat16>(p, st);
}

template <typename W>
static cudaError_t replace_by(const Replace& p, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(W);
  const int64_t rows = p.batch * p.heads;
  auto on = [](const View& v, int64_t size) { return aligned_view(View{v.data, v.batch, v.head, 0}, size); };
  const bool wide = p.capacity % kVec == 0 && on(p.score, 4) && on(p.positions, 8) && (!p.weights.data || aligned_view(p.weights, sizeof(W)));
  if (wide) return launch_clusters(replace_kernel<W, kVec>, p, rows, blocks_for(rows, p.capacity, 2048, 4), kReplaceThreads, st);
  return launch_clusters(replace_kernel<W, 1>, p, rows, blocks_for(rows, p.capacity, 512, 4), kReplaceThreads, st);
}

cudaError_t launch_replace(const Replace& p, cudaStream_t st) {
  return p.weights_dtype == kF32 ? replace_by<float>(p, st) : replace_by<__nv_bfloat16>(p, st);
}

}  // namespace tk

// A token of each row by temperature, min-p, top-k and top-p, from a given
// uniform number: a selection by weight.
//
// With z = (x - max) / T a token's weight is w = e^z = 2^-t, t = (max - x) log2(e) / T.
// Tokens stand in the selection's order (value descending, index ascending).
// All three filters keep a prefix of it, so everything is a search for the
// place where a sum over that order passes a border: the k-th token (a sum of
// ones), the token whose mass takes the prefix to top_p of what min-p and top-k
// left, and the token where it passes u times what is kept.
//
// Sums are whole numbers: a weight is 30 bits (two products of f32 give them,
// with an error of about 2^-30 of the weight) times a power of two, so that
// neither the order of the atomics nor the split of a row changes a bit, and a
// border that the sum passes far from a token's edge is passed at the same
// token as in 64 bits.  (In f32 sums, one row in some thousand of a flat
// distribution over 100000 tokens would give a neighbour of the right token.)
//
// The filter of the selection, applied to a row: a sample gives a threshold that
// some hundred tokens reach.  One pass over the row lists those (the head) and,
// where the rest can matter, adds the others (the tail) up by bins of t, 64 an octave.  The
// first block of a row's cluster then searches the head by digits of (value,
// index), or the tail: the bin where the border lies, whose tokens the blocks send
// it in a second pass.  A bin with more tokens than it can hold is narrowed by
// digits first, and a head that it cannot hold (a row of equal values) is searched
// like a tail.
//
// One GB300, inputs changing between calls; the parts by the clock of each row's first block, median row:
//   256 x 131072 f32, top_k 200, top_p, min_p  38 us (134 MB; a plain read of them takes 23): sample 6, pass 17, the blocks'
//     lists joined 1, the head's sums 2, three searches 3.5: 30, in the slowest row 35
//   96 x 131072 bf16, nucleus of 0.9  50 us: sample 4, read and counts by value 7, the values' weights 5.5, the head's
//     vectors 2, lists and bins joined 5, the head's sums 2.5, the nucleus's end 13.5, the token 1.5: 42, in the slowest row
//     51 (pass 4 more, the nucleus's end 20, the token 4)
//   37 x 100003 f32, no filter  33.5 us: sample 2.5, pass with weights 9.5, joined 5, the head's sums 2, the token 10: 30, slowest 35
//   1 x 65536 f32  12 us: sample 3, pass 2, joined 2, the head's sums 1.5, three searches 3
// A second pass over the row takes 6 of a search's 10 us in the tail.  Above kPartMost tokens each row takes two blocks or more: 96
// x 262144 bf16 with top_p 75 us in a graph, f32 121, 4 x 262144 bf16 39.
// What is once over a row is bound by instructions that are run once and fetched for it: short loops took
// less than unrolled ones all through the searches (62 -> 50 us for the nucleus).
// 256 threads of 128 registers, two blocks an SM: with 512 of 64 the searches' state went through
// the L1, and every step took 1.6 times as long.  99 KB of shared memory a block at most: from there on 28 KB of L1 are
// left instead of 60, too few for the loads under way (the first case 48 us instead of 41).
#include <cfloat>
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSub = 64;                     // bins an octave of weight
constexpr int kOctaves = 16;                 // octaves that one histogram covers
constexpr int kBins = kSub * kOctaves;
constexpr int kWindows = 3;                  // weights below 2^-48 of the largest count as zero
constexpr float kDeepest = kOctaves * kWindows;
constexpr int kHeadCap = 2240;               // tokens that the first block searches itself, of the head
constexpr int kListCap = 1536;               // and of bins
constexpr int kHead = 1024;                  // tokens that the head should have; for one top_k of all rows up to a quarter of
constexpr int kLeastHead = 128;              // that, four times the top_k
constexpr int kIndexBits = 18, kKeyBits = 32 + kIndexBits;
constexpr int kTailBits = 14;                // bits below a mass's unit that the sum behind the histogram keeps
constexpr int64_t kPartMost = 131072;         // tokens of a block's part
constexpr int kMostBlocks = 8;               // of a cluster
// bf16 values of 2^-13 to 2^9 and their negatives are counted by value first
constexpr unsigned kLeastValue = 0x3900, kValues = 0x4400 - 0x3900;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;  // of the search by digits
constexpr int kGroup = kThreads / 32;        // of the threshold: threads that form one of 32 maxima
static_assert(kTokensMaxLen <= int64_t(1) << kIndexBits, "an index fits its bits");
static_assert(kBins == 4 * kThreads && kDigits == 2 * kThreads, "bins and digits by thread");

constexpr double kLargest = 1073741822.0;    // the largest weight
// kLargest x 2^-(i/64 + 1/128): the weight in the middle of bin i of an octave.  (So every weight is below 2^30, and the
// two halves of kPartMost weights sum to less than 2^32.)
struct Middles {
  unsigned v[kSub];
};
constexpr Middles middles() {
  double root = 1.005;  // 2^(1/128): seven square roots of 2, each by Newton's steps
  double of = 2.0;
  for (int i = 0; i < 7; ++i) {
    double s = 1.2;
    for (int n = 0; n < 60; ++n) s = 0.5 * (s + of / s);
    of = s;
  }
  root = of;
  Middles m{};
  double w = kLargest / root;
  for (int i = 0; i < kSub; ++i) {
    m.v[i] = static_cast<unsigned>(w + 0.5);
    w /= root * root;
  }
  return m;
}
__constant__ Middles kMiddles = middles();

// How values become weights: t = (most - x) (hi + lo), for x >= least and not x >= below (NaN: no bound).
struct Scale {
  float most, least, below, hi, lo;
};

// round(64 t - 1/2): the bin of x, from 0 on; -1 for what has no weight (NaN and -inf among it).
constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: a sum with it is rounded to whole numbers
__device__ __forceinline__ int bin_of(float x, const Scale& s, float* depth) {
  const float d = x == s.most ? 0.0f : s.most - x;
  const float t = d * s.hi;
  *depth = t;
  if (!(x >= s.least) || x >= s.below || !(t < kDeepest)) return -1;
  return __float_as_int(fmaf(t, static_cast<float>(kSub), -0.5f) + kMagic) - __float_as_int(kMagic);
}
// The weight of x in bin j: the result times 2^-(30 + j / 64) (j / 64 a whole number), below 2^30.
__device__ __forceinline__ unsigned weight_in(float x, int j, float t, const Scale& s, const unsigned* middle) {
  const float d = x == s.most ? 0.0f : s.most - x;
  // what rounding the difference left (the two-sum of most and -x), then the product's rest
  const float bb = d - s.most;
  const float left = x == s.most ? 0.0f : (s.most - (d - bb)) - (x + bb);
  const float rest = fmaf(d, s.hi, -t) + fmaf(d, s.lo, left * s.hi);
  const float r = (fmaf(static_cast<float>(j), -1.0f / kSub, t) - 0.5f / kSub) + rest;  // |r| <= 1/128
  const float y = r * -0.69314718f;
  const float p = fmaf(y * y, fmaf(y, 1.0f / 6.0f, 0.5f), y);                          // 2^-r - 1, to y^4 / 24 < 2^-34
  const unsigned m = middle[j % kSub];
  return m + static_cast<unsigned>(__mulhi(static_cast<int>(m), __float2int_rn(p * 4294967296.0f)));
}

// (value, index) of a token as one number, the larger the earlier in the order.
__device__ __forceinline__ uint64_t token_key(float x, int index) {
  return (static_cast<uint64_t>(order_key_f32(__float_as_uint(x))) << kIndexBits) |
         static_cast<uint64_t>((1 << kIndexBits) - 1 - index);
}
// A bf16 value leaves the 16 bits under it zeros in its key, or ones where it is negative: how many of them are next below bit `at`.
template <typename T>
__device__ __forceinline__ int filled_bits(int at) {
  return sizeof(T) == 2 && at > kIndexBits && at <= kIndexBits + 16 ? at - kIndexBits : 0;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  return __uint_as_float(value_bits_f32(static_cast<uint32_t>(key >> kIndexBits)));
}
__device__ __forceinline__ int index_of(uint64_t key) {
  return (1 << kIndexBits) - 1 - static_cast<int>(key & ((1 << kIndexBits) - 1));
}

enum : int { kOpDone, kOpBins, kOpBits, kOpDigits, kOpGather };
// What the first block asks of all.
struct Order {
  Scale scale;
  int op, window;
  int from, to;           // bins [from, to) of the window,
  int from2, to2;         // and [from2, to2) behind them (gathered only)
  uint64_t mask, value;   // keys with key & mask == value
  int shift;              // digits: (key >> shift) of kDigitBits
  int unused;
  float low, high;        // no value of the first bins lies outside,
  float low2, high2;      // and none of the others outside these
};

// Tokens in no order with their masses, and the sums of those before each first digit of their keys that differs.
template <int CAP>
struct PileShared {
  uint64_t key[CAP], mass[CAP];
  uint64_t mass_before[kDigits + 1];
  unsigned count_before[kDigits + 1];
  unsigned n;       // listed (where more than CAP: not all)
  Scale scale;      // what they weigh, in the unit of a window
  int window;
  int shift;        // the first digit's place
  uint64_t above;   // the keys' common bits over it
  uint64_t total;   // mass of those with a weight, and how many
  unsigned count;
};

// All state of a block is here: what a thread keeps beside its registers goes through the little L1 that is left.
struct Shared {
  unsigned count[kBins];                 // this block's bins; a bin's mass is low + high 2^15
  alignas(16) unsigned low[kBins];
  unsigned high[kBins];
  unsigned middle[kSub];
  uint64_t warp_mass[kWarps];
  unsigned warp_count[kWarps];
  unsigned group_max[32];
  uint64_t tail;                         // this block's mass behind the window
  Order order;
  const void* row;                       // this block's part: indices begin ... end - 1 of n
  int begin, end, n;
  Scale scale;                           // of the first pass
  PileShared<kHeadCap> head;                     // (of each block its own part, then the first block's has all)
  // of the first block
  float maxes[kMostBlocks];
  uint64_t tails[kMostBlocks], ors[kMostBlocks], ands[kMostBlocks];
  // the tail: the window's bins, and sums before each
  Scale tail_scale;
  int window;
  uint64_t mass_before[kBins + 1];
  unsigned count_before[kBins + 1];
  uint64_t mass, behind;                 // of the window; behind it (kTailBits more)
  unsigned counted;
  union {
    PileShared<kListCap> list;           // bins [list_from, list_to) and, behind them, [list_from2, list_to2) of list_window
    unsigned by_value[2 * kValues];      // bf16: tokens of each value, while bins are filled
  };
  int list_window, list_from, list_to, list_from2, list_to2;
  // a crossing: the token where a sum passes a border, and the mass up to and with it
  int found;
  uint64_t found_key, found_before, found_mass;
  unsigned few, bits[4];
  int bins[2];
  uint64_t few_key[32], few_mass[32];
  float least;
  float top_p, u;
  int listed;                            // whether the head is (else all is the tail)
};
static_assert(sizeof(Shared) <= 99328, "two blocks leave 60 KB of L1");
// The block's own.  (Not handed down as a reference: the compiler has to see that it is shared memory.)
__device__ __forceinline__ Shared& own() {
  extern __shared__ __align__(16) unsigned char smem[];
  return *reinterpret_cast<Shared*>(smem);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One value for each thread of the block: sums over the threads before, and over all.
__device__ __forceinline__ void scan_before(uint64_t mass, unsigned count, uint64_t* mass_before, unsigned* count_before, uint64_t* mass_all,
                                            unsigned* count_all) {
  Shared& s = own();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint64_t m = mass;
  unsigned c = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t mo = __shfl_up_sync(~0u, m, o);
    const unsigned co = __shfl_up_sync(~0u, c, o);
    if (lane >= o) {
      m += mo;
      c += co;
    }
  }
  if (lane == 31) {
    s.warp_mass[warp] = m;
    s.warp_count[warp] = c;
  }
  __syncthreads();
  uint64_t mb = 0, ma = 0;
  unsigned cb = 0, ca = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const uint64_t mw = s.warp_mass[w];
    const unsigned cw = s.warp_count[w];
    if (w < warp) {
      mb += mw;
      cb += cw;
    }
    ma += mw;
    ca += cw;
  }
  *mass_before = mb + m - mass;
  *count_before = cb + c - count;
  *mass_all = ma;
  *count_all = ca;
  __syncthreads();
}

// 16 bytes of the row at an end of it, what is outside as -inf.
template <typename T>
__device__ __noinline__ uint4 end_of_row(const T* row, int i, int n) {
  uint32_t w[4] = {};
#pragma unroll
  for (int e = 0; e < 16 / static_cast<int>(sizeof(T)); ++e) {
    const T x = i + e >= 0 && i + e < n ? row[i + e] : from_f32<T>(-INFINITY);
    if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(x);
    else w[e / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(x)) << 16 * (e % 2);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 16 bytes of the row from value i on.
template <typename T>
__device__ __forceinline__ uint4 vector_at(int i) {
  constexpr int kVec = 16 / sizeof(T);
  const Shared& s = own();
  const T* row = static_cast<const T*>(s.row);
  return i >= 0 && i + kVec <= s.n ? ld_stream_v4(row + i) : end_of_row(row, i, s.n);
}
// f(16 bytes of values, index of the first) over the block's part of the row; what is outside the row is -inf.  After each
// kAhead of them, note(those for which f was true, index of the first) where there are any.
template <typename T, int kAhead, typename F, typename N>
__device__ __forceinline__ void each_vector(F f, N note) {
  constexpr int kVec = 16 / sizeof(T), kStep = kThreads * kVec;
  const Shared& s = own();
  const T* row = static_cast<const T*>(s.row);
  const int end = s.end, n = s.n;
  const unsigned inside = n >= kVec ? n - kVec + 1 : 0;  // first values of whole vectors
  // (each is followed by the load of the one kAhead further on, so that as many are always under way)
  int at = s.begin + threadIdx.x * kVec;
  Raw<T, kVec> raw[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a)
    if (at + a * kStep < end && static_cast<unsigned>(at + a * kStep) < inside) raw[a].u = ld_stream_v4(row + at + a * kStep);
#pragma unroll 1
  for (; at < end; at += kAhead * kStep) {
    unsigned hits = 0;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = at + a * kStep, next = i + kAhead * kStep;
      if (i >= end) break;
      if (static_cast<unsigned>(i) >= inside) raw[a].u = end_of_row(row, i, n);
      if (f(raw[a], i)) hits |= 1u << a;
      if (next < end && static_cast<unsigned>(next) < inside) raw[a].u = ld_stream_v4(row + next);
    }
    if (hits) note(hits, at);
  }
}
// Keeps the indices of noted vectors: s.few of them, those from the number `most` on not held.
template <typename T>
__device__ __forceinline__ void keep_noted(unsigned* noted, unsigned most, unsigned hits, int at) {
  constexpr int kStep = kThreads * 16 / sizeof(T);
  unsigned place = atomicAdd(&own().few, static_cast<unsigned>(__popc(hits)));
#pragma unroll 1
  for (; hits; hits &= hits - 1, ++place)
    if (place < most) noted[place] = static_cast<unsigned>(at + (__ffs(static_cast<int>(hits)) - 1) * kStep);
}
// The largest of 16 bytes of values (NaN where all are).
template <typename T>
__device__ __forceinline__ float top_of(const Raw<T, 16 / sizeof(T)>& raw) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(raw.u.x), __uint_as_float(raw.u.y)), fmaxf(__uint_as_float(raw.u.z), __uint_as_float(raw.u.w)));
  } else {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw.u);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
}

// take(value, its number) for the values of 16 bytes that are wanted: mostly one, so one at a time (eight in a row in the code, run
// once a call, took longer to fetch than to run).
template <typename T, typename W, typename F>
__device__ __forceinline__ void each_of(const Raw<T, 16 / sizeof(T)>& raw, W wanted, F take) {
  constexpr int kVec = 16 / sizeof(T);
  Vec<T, kVec> v;
  v.set_raw(raw);
  unsigned in = 0;
#pragma unroll
  for (int e = 0; e < kVec; ++e) in |= wanted(v.v[e]) ? 1u << e : 0;
#pragma unroll 1
  for (; in; in &= in - 1) {
    const int e = __ffs(static_cast<int>(in)) - 1, word = e * static_cast<int>(sizeof(T)) / 4;
    const uint32_t w = word < 2 ? word == 0 ? raw.u.x : raw.u.y : word == 2 ? raw.u.z : raw.u.w;
    take(__uint_as_float(sizeof(T) == 4 ? w : e & 1 ? w & 0xffff0000u : w << 16), e);
  }
}

template <typename T>
__device__ __forceinline__ void clear_bins() {
  Shared& s = own();
  for (int b = threadIdx.x; b < kBins; b += kThreads) s.count[b] = s.low[b] = s.high[b] = 0;
  if constexpr (sizeof(T) == 2)
    for (unsigned i = threadIdx.x; i < 2 * kValues; i += kThreads) s.by_value[i] = 0;
  if (threadIdx.x == 0) s.tail = 0;
}
// Adds `times` tokens of each value x to its bin of the window that begins `base` bins down, or to the mass behind it.  (The N
// weights are formed side by side.)
template <int N>
__device__ __forceinline__ void add_to_bins(const float* x, const unsigned* times, const Scale& scale, int base, uint64_t* tail) {
  Shared& s = own();
  int j[N];
  unsigned w[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    float t;
    j[e] = bin_of(x[e], scale, &t) - base;
    w[e] = weight_in(x[e], max(j[e] + base, 0), t, scale, s.middle);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (j[e] >= 0 && j[e] < kBins) {
      atomicAdd(&s.count[j[e]], times[e]);
      atomicAdd(&s.low[j[e]], (w[e] & 0x7fffu) * times[e]);
      atomicAdd(&s.high[j[e]], (w[e] >> 15) * times[e]);
    } else if (j[e] >= kBins) {
      const int up = kOctaves - 1 + kTailBits - j[e] / kSub;
      const uint64_t m = static_cast<uint64_t>(w[e]) * times[e];
      *tail += up >= 0 ? m << up : m >> -up;
    }
  }
}
// The bins of the block's part.  (They are clear, and the counts by value.)  A bf16 row has few values among its tokens: they
// are counted by value, one atomic each, and each value's weight is formed once.
template <typename T, typename F, typename N>
__device__ __forceinline__ void fill_bins(const Scale& scale, int base, F look, N note) {
  constexpr int kVec = 16 / sizeof(T);
  Shared& s = own();
  uint64_t tail = 0;
  if constexpr (sizeof(T) == 4) {
    each_vector<T, 3>([&](const Raw<T, kVec>& raw, int i) -> bool {
      Vec<T, kVec> v;
      v.set_raw(raw);
      const unsigned one[kVec] = {1, 1, 1, 1};
      add_to_bins<kVec>(v.v, one, scale, base, &tail);
      return look(raw, i);
    }, note);
  } else {
    each_vector<T, 2>([&](const Raw<T, kVec>& raw, int i) -> bool {
      const uint32_t w[4] = {raw.u.x, raw.u.y, raw.u.z, raw.u.w};
      uint32_t a[4], low = 0xffffffffu, high = 0;  // without signs, two a word
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q] = w[q] & 0x7fff7fffu;
        low = __vminu2(low, a[q]);
        high = __vmaxu2(high, a[q]);
      }
      low = min(low & 0xffffu, low >> 16);
      high = max(high & 0xffffu, high >> 16);
      if (low >= kLeastValue && high < kLeastValue + kValues) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // (both halves at once: below 2^16 each)
          const uint32_t at = (a[q] - kLeastValue * 0x10001u) + ((w[q] >> 15) & 0x10001u) * kValues;
          atomicAdd(&s.by_value[at & 0xffffu], 1u);
          atomicAdd(&s.by_value[at >> 16], 1u);
        }
      } else {
#pragma unroll 1
        for (int e = 0; e < kVec; ++e) {
          const uint32_t pair = e < 2 ? w[0] : e < 4 ? w[1] : e < 6 ? w[2] : w[3];
          const unsigned h = e & 1 ? pair >> 16 : pair & 0xffffu, at = (h & 0x7fffu) - kLeastValue;
          if (at < kValues) atomicAdd(&s.by_value[at + (h >> 15) * kValues], 1u);
          else {
            const float x = __uint_as_float(h << 16);
            const unsigned one = 1;
            add_to_bins<1>(&x, &one, scale, base, &tail);
          }
        }
      }
      return look(raw, i);
    }, note);
    __syncthreads();
    // (a warp takes 128 neighbouring values at a time: most such runs have tokens throughout, or none)
    constexpr unsigned kTogether = 4;
#pragma unroll 1
    for (unsigned at0 = threadIdx.x / 32 * (32 * kTogether) + threadIdx.x % 32; at0 < 2 * kValues; at0 += kTogether * kThreads) {
      float x[kTogether];
      unsigned times[kTogether], any = 0;
#pragma unroll
      for (unsigned e = 0; e < kTogether; ++e) {
        const unsigned at = at0 + e * 32;
        any |= times[e] = at < 2 * kValues ? s.by_value[at] : 0;
        // (a value without tokens has no bin)
        x[e] = times[e] ? __uint_as_float((at < kValues ? kLeastValue + at : 0x8000u + kLeastValue + at - kValues) << 16) : -INFINITY;
      }
      if (any) add_to_bins<kTogether>(x, times, scale, base, &tail);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) tail += __shfl_xor_sync(~0u, tail, d);
  if (threadIdx.x % 32 == 0 && tail) atomicAdd(reinterpret_cast<unsigned long long*>(&s.tail), static_cast<unsigned long long>(tail));
}
// Each block adds up its share of the cluster's bins and puts them into the first block's.  (After a cluster barrier.)
__device__ __forceinline__ void join_bins() {
  Shared& s = own();
  cg::cluster_group cluster = cg::this_cluster();
  Shared* first = cluster.map_shared_rank(&s, 0);
  const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
  const int share = (kBins + blocks - 1) / blocks;
  for (int b = rank * share + threadIdx.x; b < min((rank + 1) * share, kBins); b += kThreads) {
    unsigned count = 0;
    uint64_t low = 0, high = 0;
    for (int p = 0; p < blocks; ++p) {
      const Shared* peer = cluster.map_shared_rank(&s, p);
      count += peer->count[b];
      low += peer->low[b];
      high += peer->high[b];
    }
    first->mass_before[b] = low + (high << 15);
    first->count_before[b] = count;
  }
  if (threadIdx.x == 0) first->tails[rank] = s.tail;
}

// The first block's order, put into every block's memory.
__device__ __forceinline__ void tell() {
  Shared& s = own();
  static_assert(sizeof(Order) % 8 == 0, "whole words");
  constexpr int kWords = sizeof(Order) / 8;
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = static_cast<int>(cluster.num_blocks());
  if (blocks > 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < (blocks - 1) * kWords; i += kThreads)
      reinterpret_cast<uint64_t*>(&cluster.map_shared_rank(&s, 1 + i / kWords)->order)[i % kWords] = reinterpret_cast<const uint64_t*>(&s.order)[i % kWords];
  }
  cluster_sync();
}
template <bool HEAD>
__device__ __forceinline__ auto& pile(Shared& s) {
  if constexpr (HEAD) return s.head;
  else return s.list;
}
// Moves this block's part of a pile to the first block's.  (Before a cluster barrier.)
template <bool HEAD>
__device__ __forceinline__ void hand_over() {
  Shared& s = own();
  auto& from = pile<HEAD>(s);
  auto& to = pile<HEAD>(*cg::this_cluster().map_shared_rank(&s, 0));
  __syncthreads();
  if (threadIdx.x == 0) s.found = static_cast<int>(atomicAdd(&to.n, from.n));
  __syncthreads();
  constexpr unsigned kCap = HEAD ? kHeadCap : kListCap;
  const unsigned n = min(from.n, kCap), at = static_cast<unsigned>(s.found);
  for (unsigned i = threadIdx.x; i < n; i += kThreads)
    if (at + i < kCap) to.key[at + i] = from.key[i];
}

// What every block of the cluster does for the order that it holds.
template <typename T>
__device__ __noinline__ void serve() {
  constexpr int kVec = 16 / sizeof(T);
  Shared& s = own();
  const Scale scale = s.order.scale;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int op = s.order.op, base = s.order.window * kBins;
  if (op == kOpBins) {
    clear_bins<T>();
    __syncthreads();
    fill_bins<T>(scale, base, [](const Raw<T, kVec>&, int) { return false; }, [](unsigned, int) {});
    cluster_sync();
    join_bins();
  } else {
    if (rank != 0 && threadIdx.x == 0) s.list.n = 0;  // (the first block's: before the order, as others add to it)
    if (op == kOpDigits) {
      clear_bins<T>();
      __syncthreads();
    }
    const float low = s.order.low, high = s.order.high, other_low = s.order.low2, other_high = s.order.high2;
    uint64_t any = 0, none = 0;
    const int from = s.order.from, to = s.order.to, from2 = s.order.from2, to2 = s.order.to2;
    const uint64_t mask = s.order.mask, value = s.order.value;
    const int shift = s.order.shift;
    auto near = [&](float x) { return (x >= low && x <= high) || (x >= other_low && x <= other_high); };
    auto take = [&](float x, int index) {
      float t;
      const int j = bin_of(x, scale, &t) - base;
      if ((j < from || j >= to) && (j < from2 || j >= to2)) return;
      const uint64_t key = token_key(x, index);
      if ((key & mask) != value) return;
      if (op == kOpGather) {
        const unsigned at = atomicAdd(&s.list.n, 1u);
        if (at < kListCap) s.list.key[at] = key;
      } else if (op == kOpBits) {
        any |= key;
        none |= ~key;
      } else {
        const unsigned w = weight_in(x, j + base, t, scale, s.middle);
        const int digit = kDigits - 1 - static_cast<int>((key >> shift) & (kDigits - 1));
        atomicAdd(&s.count[digit], 1u);
        atomicAdd(&s.low[digit], w & 0x7fffu);
        atomicAdd(&s.high[digit], w >> 15);
      }
    };
    // 16 bytes with a value of the bins are noted first: most have none, and the rest is for whole warps then
    unsigned* noted = reinterpret_cast<unsigned*>(s.list.mass);
    constexpr unsigned kNoted = sizeof(s.list.mass) / sizeof(unsigned);
    if (threadIdx.x == 0) s.few = 0;
    __syncthreads();
    if constexpr (sizeof(T) == 4) {
      each_vector<T, 2>([&](const Raw<T, kVec>& raw, int) {
        Vec<T, kVec> v;
        v.set_raw(raw);
        bool near = false;
#pragma unroll
        for (int e = 0; e < kVec; ++e) near |= (v.v[e] >= low && v.v[e] <= high) || (v.v[e] >= other_low && v.v[e] <= other_high);
        return near;
      }, [&](unsigned hits, int at) { keep_noted<T>(noted, kNoted, hits, at); });
    } else {
      // (rounded down and up: a bf16 value is within the one bounds if it is within the others, but for some more at the ends)
      const __nv_bfloat162 low2 = __bfloat162bfloat162(__float2bfloat16_rd(low)), high2 = __bfloat162bfloat162(__float2bfloat16_ru(high));
      const __nv_bfloat162 other_low2 = __bfloat162bfloat162(__float2bfloat16_rd(other_low)), other_high2 = __bfloat162bfloat162(__float2bfloat16_ru(other_high));
      each_vector<T, 2>([&](const Raw<T, kVec>& raw, int) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw.u);
        unsigned near = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          near |= (__hge2_mask(h[q], low2) & __hle2_mask(h[q], high2)) | (__hge2_mask(h[q], other_low2) & __hle2_mask(h[q], other_high2));
        return near != 0;
      }, [&](unsigned hits, int at) { keep_noted<T>(noted, kNoted, hits, at); });
    }
    __syncthreads();
    const unsigned found = s.few;
    __syncthreads();
    auto take_all = [&](const Raw<T, kVec>& raw, int i) {
      each_of<T>(raw, near, [&](float x, int e) { take(x, i + e); });
      return false;
    };
    if (found <= kNoted) {
#pragma unroll 1
      for (unsigned q = threadIdx.x; q < found; q += kThreads) {
        Raw<T, kVec> raw;
        raw.u = vector_at<T>(static_cast<int>(noted[q]));
        take_all(raw, static_cast<int>(noted[q]));
      }
    } else {
      each_vector<T, 1>(take_all, [](unsigned, int) {});
    }
    if (op == kOpGather) {
      if (rank != 0) hand_over<false>();
    } else if (op == kOpDigits) {
      cluster_sync();
      join_bins();
    } else {
      Shared* first = cluster.map_shared_rank(&s, 0);
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        uint64_t v = which ? none : any;
#pragma unroll
        for (int d = 16; d; d >>= 1) v |= __shfl_xor_sync(~0u, v, d);
        if (threadIdx.x % 32 == 0) s.warp_mass[threadIdx.x / 32] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
          for (int w = 1; w < kWarps; ++w) v |= s.warp_mass[w];
          if (which) first->ands[rank] = ~v;
          else first->ors[rank] = v;
        }
        __syncthreads();
      }
    }
  }
  cluster_sync();
}

// ---- the first block's searches: every thread of the block calls them -----------------
// A token's mass in units of the window that begins kOctaves x window octaves down: 2^45 for its largest weight (a token of the
// head that weighs less than one unit has none, and is one of its tokens all the same).  False: it has no weight.
__device__ __forceinline__ bool mass_of(uint64_t key, const Scale& scale, int window, const unsigned* middle, uint64_t* mass) {
  const float x = value_of(key);
  float t;
  const int j = bin_of(x, scale, &t);
  *mass = j < 0 ? 0 : (static_cast<uint64_t>(weight_in(x, j, t, scale, middle)) << (kOctaves - 1)) >> (j / kSub - kOctaves * window);
  return j >= 0;
}
__device__ __forceinline__ int digit_of(uint64_t key, int at) {
  return kDigits - 1 - static_cast<int>((key >> at) & (kDigits - 1));
}
// Counts and masses by digit: three limbs of 15 bits each.
__device__ __forceinline__ void clear_digits() {
  Shared& s = own();
#pragma unroll
  for (int d = threadIdx.x; d < kDigits; d += kThreads) s.count[d] = s.low[d] = s.low[kDigits + d] = s.high[d] = 0;
}
__device__ __forceinline__ void add_digit(int d, uint64_t m) {
  Shared& s = own();
  atomicAdd(&s.count[d], 1u);
  atomicAdd(&s.low[d], static_cast<unsigned>(m) & 0x7fffu);
  atomicAdd(&s.low[kDigits + d], static_cast<unsigned>(m >> 15) & 0x7fffu);
  atomicAdd(&s.high[d], static_cast<unsigned>(m >> 30));
}
__device__ __forceinline__ uint64_t digit_mass(int d) {
  const Shared& s = own();
  return s.low[d] + (static_cast<uint64_t>(s.low[kDigits + d]) << 15) + (static_cast<uint64_t>(s.high[d]) << 30);
}

// The masses of a pile's tokens, and their sums by the first digit.  (A token without weight gets the key 0, which is no value's.)
template <bool HEAD>
__device__ __forceinline__ void prepare_pile() {
  Shared& s = own();
  auto& p = pile<HEAD>(s);
  const int lane = threadIdx.x % 32;
  const unsigned n = min(p.n, static_cast<unsigned>(HEAD ? kHeadCap : kListCap));
  const Scale scale = p.scale;
  const int window = p.window;
  uint64_t any = 0, none = 0;
  clear_digits();
  if (threadIdx.x < 4) s.bits[threadIdx.x] = 0;
#pragma unroll 1
  for (unsigned i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = p.key[i];
    uint64_t m;
    const bool weighs = mass_of(key, scale, window, s.middle, &m);
    p.mass[i] = m;
    if (!weighs) p.key[i] = 0;
    any |= weighs ? key : 0;
    none |= weighs ? ~key : 0;
  }
  const unsigned b0 = __reduce_or_sync(~0u, static_cast<unsigned>(any)), b1 = __reduce_or_sync(~0u, static_cast<unsigned>(any >> 32));
  const unsigned b2 = __reduce_or_sync(~0u, static_cast<unsigned>(none)), b3 = __reduce_or_sync(~0u, static_cast<unsigned>(none >> 32));
  __syncthreads();
  if (lane < 4) atomicOr(&s.bits[lane], lane == 0 ? b0 : lane == 1 ? b1 : lane == 2 ? b2 : b3);
  __syncthreads();
  any = (static_cast<uint64_t>(s.bits[1]) << 32) | s.bits[0];
  const uint64_t differ = any & ((static_cast<uint64_t>(s.bits[3]) << 32) | s.bits[2]);
  const int top = 64 - __clzll(static_cast<long long>(differ)), shift = top > kDigitBits ? top - kDigitBits : 0;
#pragma unroll 1
  for (unsigned i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = p.key[i];
    if (key) add_digit(digit_of(key, shift), p.mass[i]);
  }
  __syncthreads();
  const int d = 2 * threadIdx.x;
  const uint64_t m0 = digit_mass(d), m1 = digit_mass(d + 1);
  const unsigned c0 = s.count[d], c1 = s.count[d + 1];
  uint64_t mb, mass;
  unsigned cb, count;
  scan_before(m0 + m1, c0 + c1, &mb, &cb, &mass, &count);
  p.mass_before[d] = mb;
  p.mass_before[d + 1] = mb + m0;
  p.count_before[d] = cb;
  p.count_before[d + 1] = cb + c0;
  if (threadIdx.x == 0) {
    p.mass_before[kDigits] = p.total = mass;
    p.count_before[kDigits] = p.count = count;
    p.n = n;
    p.shift = shift;
    p.above = (any >> shift) & ~uint64_t(kDigits - 1);
  }
  __syncthreads();
}

// The token of a pile where the sum over its order passes `target` (below the count or mass), by digits of the keys down to 32
// tokens: found_key, and found_mass, the mass through it.
template <typename T, bool HEAD>
__device__ __forceinline__ void search_pile(bool by_count, uint64_t target) {
  Shared& s = own();
  auto& p = pile<HEAD>(s);
#pragma unroll
  for (int d = threadIdx.x; d < kDigits; d += kThreads) {
    const uint64_t m0 = p.mass_before[d], c0 = p.count_before[d];
    const uint64_t b0 = by_count ? c0 : m0, b1 = by_count ? p.count_before[d + 1] : p.mass_before[d + 1];
    if (b0 <= target && target < b1) {
      s.found = d;
      s.found_before = b0;
      s.found_mass = m0;
    }
  }
  if (threadIdx.x == 0) s.few = 0;
  __syncthreads();
  int at = p.shift;
  uint64_t before = s.found_mass;
  target -= s.found_before;
  uint64_t prefix = p.above | static_cast<uint64_t>(kDigits - 1 - s.found);
  unsigned left = p.count_before[s.found + 1] - p.count_before[s.found];
  const unsigned n = p.n;
  __syncthreads();
#pragma unroll 1
  while (left > 32) {  // (at > 0: keys differ)
    const int skip = filled_bits<T>(at);
    prefix = prefix << skip | ((prefix >> (kKeyBits - 1 - at) & 1) ? 0 : (uint64_t(1) << skip) - 1);
    at -= skip;
    const int next = at > kDigitBits ? at - kDigitBits : 0;
    clear_digits();
    __syncthreads();
#pragma unroll 1
    for (unsigned i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t m = p.mass[i], key = p.key[i];
      if (key && key >> at == prefix) add_digit(digit_of(key, next), m);
    }
    __syncthreads();
    const int d = 2 * threadIdx.x;
    const uint64_t m0 = digit_mass(d), m1 = digit_mass(d + 1);
    const unsigned c0 = s.count[d], c1 = s.count[d + 1];
    uint64_t mb, ma;
    unsigned cb, ca;
    scan_before(m0 + m1, c0 + c1, &mb, &cb, &ma, &ca);
    const uint64_t f0 = by_count ? cb : mb, f1 = f0 + (by_count ? c0 : m0), f2 = f1 + (by_count ? c1 : m1);
    if (f0 <= target && target < f2) {
      const bool second = f1 <= target;
      s.found = d + second;
      s.found_before = second ? f1 : f0;
      s.found_mass = second ? mb + m0 : mb;
    }
    __syncthreads();
    before += s.found_mass;
    target -= s.found_before;
    left = s.count[s.found];
    // (the digit's bits above `at` are the prefix's own)
    prefix = prefix << (at - next) | (static_cast<uint64_t>(kDigits - 1 - s.found) & ((uint64_t(1) << (at - next)) - 1));
    at = next;
    __syncthreads();
  }
#pragma unroll 1
  for (unsigned i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t m = p.mass[i], key = p.key[i];
    if (key && key >> at == prefix) {
      const unsigned f = atomicAdd(&s.few, 1u);
      if (f < 32) {
        s.few_key[f] = key;
        s.few_mass[f] = m;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const unsigned few = min(s.few, 32u);
    const uint64_t key = threadIdx.x < few ? s.few_key[threadIdx.x] : 0, m = threadIdx.x < few ? s.few_mass[threadIdx.x] : 0;
    uint64_t mb = 0, cb = 0;
#pragma unroll 4
    for (unsigned f = 0; f < few; ++f) {
      const bool earlier = s.few_key[f] > key;
      mb += earlier ? s.few_mass[f] : 0;
      cb += earlier;
    }
    const uint64_t f0 = by_count ? cb : mb, f1 = by_count ? cb + 1 : mb + m;
    if (key && f0 <= target && target < f1) {
      s.found_key = key;
      s.found_mass = before + mb + m;
    }
  }
  __syncthreads();
}

// a b / 2^shift, rounded down, for results below 2^64.
__device__ __forceinline__ uint64_t scaled(uint64_t a, uint64_t b, int shift) {
  const uint64_t low = a * b, high = __umul64hi(a, b);
  if (shift <= 0) return low << -shift;
  if (shift < 64) return low >> shift | high << (64 - shift);
  return shift < 128 ? high >> (shift - 64) : 0;
}
// f a for f in (0, 1), rounded down; below: the largest whole number that is less.
__device__ __forceinline__ uint64_t share_of(float f, uint64_t a, bool below) {
  const unsigned bits = __float_as_uint(f), e = bits >> 23;
  const unsigned m = e ? (bits & 0x7fffffu) | 0x800000u : bits;
  const int shift = e ? 150 - static_cast<int>(e) : 149;
  if (!below) return scaled(a, m, shift);
  // (a m - 1) / 2^shift
  const uint64_t low = a * m, high = __umul64hi(a, m) - (low == 0), less = low - 1;
  if (shift < 64) return less >> shift | high << (64 - shift);
  return shift < 128 ? high >> (shift - 64) : 0;
}
// The tail's masses in the head's unit: times weight / 2^(30 + depth), rounded down.
struct Unit {
  unsigned weight, inverse;  // (2^54 / weight, rounded down)
  int depth;
  __device__ __forceinline__ uint64_t in_head(uint64_t m) const { return scaled(m, weight, 30 + depth); }
  __device__ __forceinline__ uint64_t in_tail(uint64_t m) const {
    const uint64_t a = scaled(m, inverse, 24 - depth), left = m - min(m, in_head(a));
    return a + scaled(left, inverse, 24 - depth);
  }
};

template <typename T>
__device__ __noinline__ void ask(int op, int w, int from, int to, uint64_t mask, uint64_t value, int shift, int from2 = 0, int to2 = 0) {
  Shared& s = own();
  if (threadIdx.x == 0) {
    // a hundredth of a bin is left at either end, and room for the differences' rounding
    const Scale scale = s.tail_scale;
    const float d = fabsf(scale.most) * 0x1p-20f, bin = 1.0f / kSub / scale.hi;
    const bool sure = fabsf(scale.most) < FLT_MAX;
    auto lowest = [&](int t) { return sure ? scale.most - (static_cast<float>(w * kBins + t) + 0.01f) * bin - d : -FLT_MAX; };
    auto highest = [&](int f) { return sure && f > 0 ? scale.most - (static_cast<float>(w * kBins + f) - 0.01f) * bin + d : INFINITY; };
    if (op == kOpBins) s.list_window = -1;
    if (op == kOpGather) s.list.n = 0;
    s.order = Order{scale, op, w, from, to, from2, to2, mask, value, shift, 0, lowest(to), highest(from),
                    from2 < to2 ? lowest(to2) : INFINITY, from2 < to2 ? highest(from2) : -INFINITY};
  }
  tell();
  serve<T>();
}
// Sums before each bin, from the bins' own.
__device__ __noinline__ void add_up_bins() {
  Shared& s = own();
  constexpr int kEach = kBins / kThreads;
  const int b = kEach * threadIdx.x;
  uint64_t m[kEach], sum = 0, mb, mass;
  unsigned c[kEach], number = 0, cb, count;
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    sum += m[q] = s.mass_before[b + q];
    number += c[q] = s.count_before[b + q];
  }
  scan_before(sum, number, &mb, &cb, &mass, &count);
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    s.mass_before[b + q] = mb;
    s.count_before[b + q] = cb;
    mb += m[q];
    cb += c[q];
  }
  if (threadIdx.x == 0) {
    s.mass_before[kBins] = s.mass = mass;
    s.count_before[kBins] = s.counted = count;
  }
  __syncthreads();
}
// Takes the bins that the blocks have joined as window w's: they hold sums of 30-bit weights, a mass is that at the octave's place.
__device__ __noinline__ void take_window(int w) {
  Shared& s = own();
  constexpr int kEach = kBins / kThreads;  // (the bins that this thread then adds up)
#pragma unroll
  for (int q = 0; q < kEach; ++q) s.mass_before[kEach * threadIdx.x + q] <<= kOctaves - 1 - (kEach * threadIdx.x + q) / kSub;
  if (threadIdx.x == 0) {
    uint64_t tail = 0;
    const int blocks = static_cast<int>(cg::this_cluster().num_blocks());
    for (int q = 0; q < blocks; ++q) tail += s.tails[q];
    s.behind = tail;
    s.window = w;
  }
  add_up_bins();
}
template <typename T>
__device__ __noinline__ void need_window(int w) {
  if (own().window == w) return;
  ask<T>(kOpBins, w, 0, kBins, 0, 0, 0);
  take_window(w);
}
// The bins (or digits) where the sums before pass N targets.
template <int N>
__device__ __noinline__ void find_bins(bool by_count, const uint64_t (&target)[N], int (&bin)[N]) {
  Shared& s = own();
#pragma unroll
  for (int b = threadIdx.x; b < kBins; b += kThreads) {
    const uint64_t b0 = by_count ? s.count_before[b] : s.mass_before[b], b1 = by_count ? s.count_before[b + 1] : s.mass_before[b + 1];
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (b0 <= target[q] && target[q] < b1) s.bins[q] = b;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < N; ++q) bin[q] = s.bins[q];
  __syncthreads();
}
__device__ __forceinline__ int find_bin(bool by_count, uint64_t target) {
  const uint64_t t[1] = {target};
  int b[1];
  find_bins<1>(by_count, t, b);
  return b[0];
}

// The token of bin b of the window where the sum passes `target`, as search_pile; masses in the window's unit.  Bins [also,
// also_to) before b are listed with it where there is room: the next search's; where that is not `known`, all before b.
template <typename T>
__device__ __forceinline__ void search_bin(int b, bool by_count, uint64_t target, bool known, int also, int also_to) {
  Shared& s = own();
  const int w = s.window, up = kOctaves - 1 - b / kSub;
  uint64_t start;                        // mass before the list
  if (s.list_window == w && b >= s.list_from && b < s.list_to) {
    start = s.mass_before[s.list_from];
    target -= by_count ? s.count_before[s.list_from] : start;
  } else if (s.list_window == w && b >= s.list_from2 && b < s.list_to2) {
    const int f = s.list_from, t = s.list_to, f2 = s.list_from2;
    start = s.mass_before[f2] - (s.mass_before[t] - s.mass_before[f]);
    target -= by_count ? s.count_before[f2] - (s.count_before[t] - s.count_before[f]) : start;
  } else {
    const int from = known || s.count_before[b + 1] > kListCap ? b : 0;
    unsigned held = s.count_before[b + 1] - s.count_before[from];
    uint64_t mask = 0, value = 0;
    start = s.mass_before[from];
    if (from == 0 || s.count_before[also_to] - s.count_before[also] + held > kListCap) also = also_to = 0;
    if (also < also_to) start -= s.mass_before[also_to] - s.mass_before[also];
    target -= by_count ? s.count_before[from] - (s.count_before[also_to] - s.count_before[also]) : start;
    if (held > kListCap) {
      // narrowed by digits over the cluster: the window's sums are made anew afterwards
      ask<T>(kOpBits, w, b, b + 1, 0, 0, 0);
      uint64_t any = 0, all = ~uint64_t(0);
      const int blocks = static_cast<int>(cg::this_cluster().num_blocks());
      for (int q = 0; q < blocks; ++q) {
        any |= s.ors[q];
        all &= s.ands[q];
      }
      int top = 64 - __clzll(static_cast<long long>(any ^ all));
      mask = ~((uint64_t(1) << top) - 1);
      value = all & mask;
      if (!by_count) target >>= up;      // (in 30-bit weights)
      uint64_t past = 0;
#pragma unroll 1
      while (held > kListCap) {
        const int skip = filled_bits<T>(top);
        top -= skip;
        const uint64_t filled = ((uint64_t(1) << skip) - 1) << top;
        mask |= filled;
        if (!(value >> (kKeyBits - 1) & 1)) value |= filled;
        const int shift = top > kDigitBits ? top - kDigitBits : 0;
        ask<T>(kOpDigits, w, b, b + 1, mask, value, shift);
        add_up_bins();
        const int digit = find_bin(by_count, target);
        held = s.count_before[digit + 1] - s.count_before[digit];
        past += s.mass_before[digit];
        target -= by_count ? s.count_before[digit] : s.mass_before[digit];
        // (digits below bit `shift` are still open; the digit's own bits above `top` are the mask's)
        const uint64_t bits = static_cast<uint64_t>(kDigits - 1 - digit) << shift;
        value = (value & mask) | (bits & ~mask);
        mask = ~((uint64_t(1) << shift) - 1);
        value &= mask;
        top = shift;
        __syncthreads();
      }
      start += past << up;
      if (!by_count) target <<= up;
      if (threadIdx.x == 0) s.window = -1;
    }
    if (also < also_to) ask<T>(kOpGather, w, also, also_to, mask, value, 0, from, b + 1);
    else ask<T>(kOpGather, w, from, b + 1, mask, value, 0);
    if (threadIdx.x == 0) {
      s.list_window = mask ? -1 : w;
      s.list_from = also < also_to ? also : from;
      s.list_to = also < also_to ? also_to : b + 1;
      s.list_from2 = also < also_to ? from : 0;
      s.list_to2 = also < also_to ? b + 1 : 0;
      s.list.scale = s.tail_scale;
      s.list.window = w;
    }
    __syncthreads();
    prepare_pile<false>();
  }
  search_pile<T, false>(by_count, target);
  if (threadIdx.x == 0) s.found_mass += start;
}

// The token where the sum over the tail passes `target`; masses in the unit of window 0.  False where it does not.  `ahead`: what
// is kept ends here, and the token is searched next, whose bin is known but for one or two: they are listed too.
template <typename T>
__device__ __forceinline__ bool search_tail(bool by_count, uint64_t target, bool ahead, const Unit& unit) {
  Shared& s = own();
  uint64_t done = 0;  // mass of the windows before
#pragma unroll 1
  for (int w = 0; w < kWindows; ++w) {
    need_window<T>(w);
    uint64_t t = by_count ? target : (target - done) << (kOctaves * w);
    const uint64_t all = by_count ? s.counted : s.mass;
    const bool last = s.behind == 0;
    if (t >= all && last && !by_count && all) t = all - 1;  // (sums of different units, rounded: the last token)
    if (t < all) {
      const int b = find_bin(by_count, t);
      int also = 0, also_to = 0;
      if (ahead && w == 0) {
        // u of what is kept, that being between the masses before and behind the bin
        const uint64_t head = s.listed ? s.head.total : 0;
        const float u = s.u > 0.0f ? fminf(s.u, 0x1.fffffep-1f) : 0.0f;
        const uint64_t low = share_of(u, head + unit.in_head(s.mass_before[b]), false), high = share_of(u, head + unit.in_head(s.mass_before[b + 1]), false);
        if (low >= head) {
          const uint64_t ends[2] = {unit.in_tail(low - head), unit.in_tail(high - head)};
          int bins[2];
          find_bins<2>(false, ends, bins);
          also = min(bins[0], b);
          also_to = min(bins[1] + 1, b);
        }
      }
      search_bin<T>(b, by_count, t, ahead && w == 0, also, also_to);
      if (threadIdx.x == 0) s.found_mass = done + (s.found_mass >> (kOctaves * w));
      __syncthreads();
      return true;
    }
    if (last) break;
    if (by_count) target -= s.counted;
    done += s.mass >> (kOctaves * w);
    if (!by_count && target < done) target = done;
  }
  return false;
}

// The block's part of the row, read once: its maximum, its part of the head, and, where `rest`, its bins.
template <typename T>
__device__ __noinline__ float first_pass(bool rest) {
  constexpr int kVec = 16 / sizeof(T);
  Shared& s = own();
  const Scale scale = s.scale;
  const float tau = scale.most;
  float most = -INFINITY;
  // 16 bytes with a token of the head are noted, and gone through again afterwards: some hundred among thousands
  unsigned* noted = reinterpret_cast<unsigned*>(s.head.mass);
  constexpr unsigned kNoted = sizeof(s.head.mass) / sizeof(unsigned);
  auto look = [&](const Raw<T, kVec>& raw, int) {
    const float top = top_of<T>(raw);
    most = fmaxf(most, top);
    return top >= tau;
  };
  auto note = [&](unsigned hits, int at) { keep_noted<T>(noted, kNoted, hits, at); };
  if (rest) fill_bins<T>(scale, 0, look, note);
  else each_vector<T, 12>(look, note);
  __syncthreads();
  const unsigned found = s.few;
  if (found > kNoted) {
    if (threadIdx.x == 0) atomicAdd(&s.head.n, kHeadCap + 1u);  // (too many)
  } else {
#pragma unroll 1
    for (unsigned q = threadIdx.x; q < found; q += kThreads) {
      const int i = static_cast<int>(noted[q]);
      Raw<T, kVec> raw;
      raw.u = vector_at<T>(i);
      each_of<T>(raw, [&](float x) { return x >= tau; }, [&](float x, int e) {
        const unsigned at = atomicAdd(&s.head.n, 1u);
        if (at < kHeadCap) s.head.key[at] = token_key(x, i + e);
      });
    }
  }
  return most;
}

// `slots`: tokens of a block's part; `head`: those that the head should have; the threshold is number `order` of the 32 maxima of `runs` times kGroup tokens each,
// `step_` apart (runs == 0: none).
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) token_kernel(const TokenDraw p, int slots, int head, int runs, int order, int step_) {
  constexpr int kVec = 16 / sizeof(T);
  Shared& s = own();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = blockIdx.x / blocks;
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  if (threadIdx.x < kSub) s.middle[threadIdx.x] = kMiddles.v[threadIdx.x];
  if (threadIdx.x == 0) {
    s.found = 0;
    s.few = 0;
    s.head.n = 0;
    s.window = s.list_window = -1;
    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) % kVec);
    s.row = x;
    s.begin = rank * slots - lead;
    s.end = min((rank + 1) * slots - lead, p.n);
    s.n = p.n;
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (threadIdx.x == 32) {
    s.u = p.u[row];
    s.top_p = p.top_ps ? p.top_ps[row] : p.top_p;
    s.least = p.min_ps ? p.min_ps[row] : p.min_p;
  }

  const float temperature = p.temperatures ? p.temperatures[row] : p.temperature;
  const bool greedy = !(temperature > 0.0f);
  const int top_k = greedy ? 1 : p.top_ks ? p.top_ks[row] : p.top_k;
  const bool rest = runs > 0 && !(top_k > 0 && top_k <= head / 4);  // (the tail is empty, or will hardly matter, otherwise)

  if (rest) clear_bins<T>();

  // the threshold: the same in all blocks of the cluster
  float tau = -FLT_MAX;
  if (runs > 0) {
    float top = -INFINITY;
    const int group = threadIdx.x / kGroup;
#pragma unroll 8
    for (int i = 0; i < runs; ++i) top = fmaxf(top, to_f32(x[(i * 32 + group) * step_ + threadIdx.x % kGroup]));
#pragma unroll
    for (int d = kGroup / 2; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (threadIdx.x % kGroup == 0) s.group_max[group] = __float_as_uint(top);
    __syncthreads();
    top = __uint_as_float(s.group_max[lane]);
    int place = 0;
#pragma unroll 8
    for (int q = 0; q < 32; ++q) {
      const float other = __shfl_sync(~0u, top, q);
      place += other > top || (other == top && q < lane);
    }
    top = __shfl_sync(~0u, top, __ffs(static_cast<int>(__ballot_sync(~0u, place == order))) - 1);
    if (top > -INFINITY) tau = top;
  }
  if (threadIdx.x == 0) {
    const double per = greedy ? INFINITY : p.temperatures ? 1.4426950408889634 / static_cast<double>(temperature) : p.per;  // log2(e) / T
    const bool within = per < FLT_MAX;
    const float hi = within ? static_cast<float>(per) : FLT_MAX;
    s.scale = Scale{tau, -FLT_MAX, tau, hi, within ? static_cast<float>(per - static_cast<double>(hi)) : 0.0f};
  }
  cluster_sync();  // (every block has started, with nothing in its lists)

  float most = first_pass<T>(rest);
#pragma unroll
  for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
  if (lane == 0) s.warp_count[warp] = __float_as_uint(most);
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) most = fmaxf(most, __uint_as_float(s.warp_count[w]));
    cluster.map_shared_rank(&s, 0)->maxes[rank] = most;
  }
  if (rank != 0) hand_over<true>();
  cluster_sync();
  if (rest) {
    join_bins();
    cluster_sync();
  }
  if (rank != 0) {
#pragma unroll 1
    for (;;) {
      cluster_sync();
      if (s.order.op == kOpDone) return;
      serve<T>();
    }
  }

  most = s.maxes[0];
  for (int b = 1; b < blocks; ++b) most = fmaxf(most, s.maxes[b]);
  const bool listed = s.head.n <= kHeadCap;
  const Scale scale = s.scale;
  __syncthreads();
  if (threadIdx.x == 0) {
    float least = -FLT_MAX;
    const float min_p = s.least;
    if (greedy) {
      least = most;
    } else if (min_p > 0.0f) {  // w >= min_p: x >= max + T ln(min_p)
      const double depth = p.min_ps ? log(static_cast<double>(min_p)) : p.log_min_p;
      const float f = __double2float_ru(static_cast<double>(most) + static_cast<double>(temperature) * depth);
      least = fminf(fmaxf(f, -FLT_MAX), most);
    }
    s.least = least;
    s.listed = listed;
    s.tail_scale = listed ? Scale{tau, least, tau, scale.hi, scale.lo} : Scale{most, least, NAN, scale.hi, scale.lo};
    s.head.scale = Scale{most, least, NAN, scale.hi, scale.lo};
    s.head.window = 0;
    if (!listed) s.head.n = 0;
  }
  __syncthreads();
  // the tail's unit: the weight of its largest value
  Unit unit{1u << 30, 1u << 24, 0};
  bool more = true;
  if (listed) {
    float t;
    const Scale from{most, -FLT_MAX, NAN, scale.hi, scale.lo};
    const int j = bin_of(tau, from, &t);
    more = j >= 0 && s.least < tau;
    if (more) {
      const unsigned w = weight_in(tau, j, t, from, s.middle);
      unit = Unit{w + ((w + (1u << 28)) >> 29), 0, j / kSub};  // (w / kLargest 2^30)
      unit.inverse = __float2uint_rd(__frcp_rd(__uint2float_ru(unit.weight)) * 0x1p54f) - 2;
    }
  }
  bool found = false;
  uint64_t kept = 0;
  if (most > -INFINITY) {  // (else nothing may be drawn)
    if (listed && more && rest && s.least == -FLT_MAX) take_window(0);
    prepare_pile<true>();
    const uint64_t head_mass = s.head.total;
    const unsigned head_count = s.head.count;
    // in steps: the first top_k tokens, or all; what top_p leaves of them; the token
    bool in_head = true;
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
      uint64_t target = ~uint64_t(0);  // (no border)
      if (step == 0) {
        in_head = static_cast<unsigned>(top_k) <= head_count;
        if (top_k > 0 && top_k < p.n && (in_head || more)) target = static_cast<uint64_t>(top_k - 1) - (in_head ? 0 : head_count);
      } else {
        const float f = step == 2 ? s.u : s.top_p;
        if (step == 1 && !(f < 1.0f)) continue;
        target = !(f > 0.0f) ? 0 : f < 1.0f ? share_of(f, kept, step == 1) : kept - 1;
        in_head = !more || (listed && target < head_mass);
        target = in_head ? min(target, head_mass - 1) : unit.in_tail(target - head_mass);
      }
      found = false;
      if (target != ~uint64_t(0)) {
        if (!in_head) found = search_tail<T>(step == 0, target, step == 1, unit);
        if (!found && (in_head || (step && listed))) {
          search_pile<T, true>(step == 0, in_head ? target : head_mass - 1);
          in_head = found = true;
        }
      }
      if (step == 2) break;
      if (found) {
        const uint64_t through = in_head ? s.found_mass : head_mass + unit.in_head(s.found_mass);
        kept = step ? min(kept, through) : through;
      } else if (step == 0) {
        kept = head_mass;
        if (more) {
          need_window<T>(0);
          kept += unit.in_head(s.mass + (s.behind >> kTailBits));
        }
      }
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) {
    p.tokens[row] = found ? index_of(s.found_key) : -1;
    // z - ln(kept), with z = -t ln 2 in two parts
    const float x0 = value_of(s.found_key);
    const float d = x0 == most ? 0.0f : most - x0, bb = d - most, left = x0 == most ? 0.0f : (most - (d - bb)) - (x0 + bb);
    const float t = d * scale.hi, more_t = fmaf(d, scale.hi, -t) + fmaf(d, scale.lo, left * scale.hi);
    const float z = greedy ? 0.0f : t * 0.693147182f;
    const float low = greedy ? 0.0f : fmaf(t, 0.693147182f, -z) + fmaf(more_t, 0.693147182f, t * -1.90465421e-9f);
    const uint64_t one = static_cast<uint64_t>(kLargest) << (kOctaves - 1);
    const float share = greedy ? 0.0f : log1pf(static_cast<float>(kept > one ? kept - one : 0) * static_cast<float>(0x1p-15 / kLargest));
    p.logprobs[row] = found ? 0.0f - static_cast<float>(static_cast<double>(z) + low + share) : -INFINITY;
    s.order.op = kOpDone;
  }
  tell();
}

}  // namespace

static cudaLaunchConfig_t config(int blocks, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of that many blocks that the device runs at once (a cluster's blocks lie on neighbouring SMs: 37 of eight blocks, two an
// SM, took two rounds on 152 SMs).
template <typename T>
static int clusters_at_once(int blocks) {
  static PerDevice known[kMostBlocks + 1];
  std::atomic<int>* k = known[blocks].here();
  int n = k ? k->load() : 0;
  if (n) return n;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(blocks, attr);
  if (cudaOccupancyMaxActiveClusters(&n, token_kernel<T>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 1;
  }
  if (k) *k = n;
  return n;
}

template <typename T>
static cudaError_t launch(const TokenDraw& p, cudaStream_t st) {
  constexpr int64_t kVec = 16 / sizeof(T);
  // blocks a row: as many as let all rows' clusters run at once, down to 2048 tokens each
  const int64_t len = p.n + kVec, least = p.n <= kPartMost ? 1 : (len - 1) / (kPartMost - kVec) + 1;  // (parts are whole vectors)
  cudaError_t e = cudaFuncSetAttribute(token_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
  if (e != cudaSuccess) return e;
  int64_t blocks = 2 * ops_sm_count() / p.rows;
  if (blocks > len / 2048) blocks = len / 2048;
  blocks = blocks < least ? least : blocks > kMostBlocks ? kMostBlocks : blocks;
  while (blocks > least && clusters_at_once<T>(static_cast<int>(blocks)) < p.rows) --blocks;
  const int64_t slots = ((len + blocks - 1) / blocks + kVec - 1) / kVec * kVec;
  if (p.rows * blocks > INT32_MAX) return cudaErrorNotSupported;
  // the threshold: of 32 maxima of m tokens each, number i (from 0) has about (1/32 + ... + 1/(32 - i)) n / m tokens above it
  int runs = 0, order = 0;
  int head = kHead;
  if (!p.top_ks && p.top_k > 0 && p.top_k < kHead / 4) head = 4 * p.top_k > kLeastHead ? 4 * p.top_k : kLeastHead;
  if (p.n > kHeadCap) {
    runs = static_cast<int>((static_cast<int64_t>(p.n) * 69 / 100 / head + kGroup - 1) / kGroup);
    double above = 1.0 / 32;
    while (order < 31 && above * p.n < 1.0 * kGroup * runs * head) above += 1.0 / (32 - ++order);
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(static_cast<int>(blocks), attr);
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows * blocks));
  cfg.stream = st;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_kernel<T>, p, static_cast<int>(slots), head, runs, order,
                            runs ? (p.n - kGroup) / (32 * runs) : 0);
}

cudaError_t launch_tokens(const TokenDraw& p, cudaStream_t st) {
  return p.dtype == kF32 ? launch<float>(p, st) : launch<__nv_bfloat16>(p, st);
}

}  // namespace tk

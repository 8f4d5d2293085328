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
// A cluster holds a row in its shared memory, a part a block, and reads it from
// memory once.  Bins of t (64 an octave, 16 octaves at a time) take the counts and
// masses; the first block of the cluster adds them up, finds the bin where the
// border lies, has the others send it the tokens of that bin (or of all bins up to
// it where those are few) and finds the token among them by digits of (value,
// index).  A bin with more tokens than it can hold is narrowed by digits over the cluster first.
#include <cfloat>
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "ops_common.cuh"

namespace tk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSub = 64;                     // bins an octave of weight
constexpr int kOctaves = 16;                 // octaves that one histogram covers
constexpr int kBins = kSub * kOctaves;
constexpr int kWindows = 3;                  // weights below 2^-48 of the largest count as zero
constexpr float kDeepest = kOctaves * kWindows;
constexpr int kCap = 2048;                   // tokens that the first block searches itself
constexpr int kEach = kCap / kThreads;
constexpr int kIndexBits = 18;
constexpr int kTailBits = 14;                // bits below a mass's unit that the sum behind the histogram keeps
constexpr int kDigitBits = 9;                // of the search by digits: a bin a thread
static_assert(kTokensMaxLen <= int64_t(1) << kIndexBits, "an index fits its bits");
static_assert(kBins == 2 * kThreads && (1 << kDigitBits) == kThreads, "bins by thread");

// 2^30 x 2^-(i/64 + 1/128): the weight in the middle of bin i of an octave.
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
  double w = 1073741824.0 / root;
  for (int i = 0; i < kSub; ++i) {
    m.v[i] = static_cast<unsigned>(w + 0.5);
    w /= root * root;
  }
  return m;
}
__constant__ Middles kMiddles = middles();

// How a row's values become weights: t = (most - x) (hi + lo), for x >= least.
struct Scale {
  float most, least, hi, lo;
};

// round(64 t - 1/2): the bin of x, from 0 on; -1 for what has no weight (NaN and -inf among it).
constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: a sum with it is rounded to whole numbers
__device__ __forceinline__ int bin_of(float x, const Scale& s, float* depth) {
  const float d = x == s.most ? 0.0f : s.most - x;
  const float t = d * s.hi;
  *depth = t;
  if (!(x >= s.least) || !(t < kDeepest)) return -1;
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
__device__ __forceinline__ float value_of(uint64_t key) {
  return __uint_as_float(value_bits_f32(static_cast<uint32_t>(key >> kIndexBits)));
}
__device__ __forceinline__ int index_of(uint64_t key) {
  return (1 << kIndexBits) - 1 - static_cast<int>(key & ((1 << kIndexBits) - 1));
}

enum : int { kOpDone, kOpBins, kOpBits, kOpDigits, kOpGather };
// What the first block asks of all.
struct Order {
  int op, window;
  int from, to;           // bins [from, to) of the window
  uint64_t mask, value;   // keys with key & mask == value
  int shift;              // digits: (key >> shift) of kDigitBits
};

struct Shared {
  unsigned count[kBins], low[kBins], high[kBins];  // this block's; a bin's mass is low + high 2^15
  unsigned middle[kSub];
  float maxes[16];            // of each block, in every block
  uint64_t warp_mass[kWarps];
  unsigned warp_count[kWarps];
  uint64_t tail;              // this block's mass behind the window
  Order order;
  // of the first block
  uint64_t mass_before[kBins + 1];
  unsigned count_before[kBins + 1];
  uint64_t tails[16], ors[16], ands[16];
  uint64_t list[kCap];
  unsigned listed;
  int found;
  uint64_t found_key;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One value for each thread of the block: sums over the threads before.
__device__ __forceinline__ void scan_before(Shared& s, uint64_t mass, unsigned count, uint64_t* mass_before, unsigned* count_before,
                                            uint64_t* mass_all, unsigned* count_all) {
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

template <typename T>
struct Part {        // this block's part of the row
  const T* data;     // shared memory; what is outside the row is -inf
  int slots;         // multiple of a vector
  int index0;        // index in the row of slot 0 (may be negative)
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int kVec = 16 / sizeof(T);
    for (int at = threadIdx.x * kVec; at < slots; at += kThreads * kVec) {
      Vec<T, kVec> v;
      v.load(data + at);
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(v.v[e], index0 + at + e);
    }
  }
};

// What every block of the cluster does for one order; `first`: the first block's shared memory.
template <typename T>
__device__ void serve(Shared& s, Shared& first, cg::cluster_group& cluster, const Order& o, const Part<T>& part, const Scale& scale) {
  const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
  const int lane = threadIdx.x % 32;
  const int base = o.window * kBins;
  if (o.op == kOpBins || o.op == kOpDigits) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) s.count[b] = s.low[b] = s.high[b] = 0;
    if (threadIdx.x == 0) s.tail = 0;
    __syncthreads();
    uint64_t tail = 0;
    part.each([&](float x, int index) {
      float t;
      const int j = bin_of(x, scale, &t) - base;
      if (o.op == kOpBins) {
        if (j < 0 || t >= kDeepest) return;
        const unsigned w = weight_in(x, j + base, t, scale, s.middle);
        if (j < kBins) {
          atomicAdd(&s.count[j], 1u);
          atomicAdd(&s.low[j], w & 0x7fffu);
          atomicAdd(&s.high[j], w >> 15);
        } else {
          const int up = kOctaves - 1 + kTailBits - j / kSub;
          tail += up >= 0 ? static_cast<uint64_t>(w) << up : w >> -up;
        }
      } else if (j >= o.from && j < o.to) {
        const uint64_t key = token_key(x, index);
        if ((key & o.mask) != o.value) return;
        const unsigned w = weight_in(x, j + base, t, scale, s.middle);
        const int digit = (1 << kDigitBits) - 1 - static_cast<int>((key >> o.shift) & ((1 << kDigitBits) - 1));
        atomicAdd(&s.count[digit], 1u);
        atomicAdd(&s.low[digit], w & 0x7fffu);
        atomicAdd(&s.high[digit], w >> 15);
      }
    });
    if (o.op == kOpBins) {
#pragma unroll
      for (int d = 16; d; d >>= 1) tail += __shfl_xor_sync(~0u, tail, d);
      if (lane == 0 && tail) atomicAdd(reinterpret_cast<unsigned long long*>(&s.tail), static_cast<unsigned long long>(tail));
    }
    cluster_sync();
    // each block adds up its share of the bins and puts them into the first block's
    const int share = kBins / blocks;
    for (int b = rank * share + threadIdx.x; b < (rank + 1) * share; b += kThreads) {
      unsigned count = 0;
      uint64_t low = 0, high = 0;
      for (int p = 0; p < blocks; ++p) {
        const Shared* peer = cluster.map_shared_rank(&s, p);
        count += peer->count[b];
        low += peer->low[b];
        high += peer->high[b];
      }
      first.mass_before[b] = low + (high << 15);
      first.count_before[b] = count;
    }
    if (threadIdx.x == 0) first.tails[rank] = s.tail;
  } else if (o.op == kOpBits) {
    uint64_t any = 0, all = ~uint64_t(0);
    part.each([&](float x, int index) {
      float t;
      const int j = bin_of(x, scale, &t) - base;
      if (j < o.from || j >= o.to) return;
      const uint64_t key = token_key(x, index);
      any |= key;
      all &= key;
    });
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      any |= __shfl_xor_sync(~0u, any, d);
      all &= __shfl_xor_sync(~0u, all, d);
    }
    __syncthreads();
    if (lane == 0) s.warp_mass[threadIdx.x / 32] = any;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 1; w < kWarps; ++w) any |= s.warp_mass[w];
    __syncthreads();
    if (lane == 0) s.warp_mass[threadIdx.x / 32] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) all &= s.warp_mass[w];
      first.ors[rank] = any;
      first.ands[rank] = all;
    }
  } else if (o.op == kOpGather) {
    part.each([&](float x, int index) {
      float t;
      const int j = bin_of(x, scale, &t) - base;
      if (j < o.from || j >= o.to) return;
      const uint64_t key = token_key(x, index);
      if ((key & o.mask) != o.value) return;
      const unsigned at = atomicAdd(&first.listed, 1u);
      if (at < kCap) first.list[at] = key;
    });
  }
  cluster_sync();
}

// Where a sum over the order passes a border: the token, and the mass up to and with it (in the unit of window 0).
struct Crossing {
  bool found;
  uint64_t key, through;
};

// The first block's search.  Every thread of the block calls its functions and has the same results.
template <typename T>
struct Search {
  Shared& s;
  cg::cluster_group& cluster;
  const Part<T>& part;
  const Scale& scale;
  int window;                          // the bins in s are this window's
  uint64_t mass;                       // of the window
  unsigned count;
  uint64_t tail;                       // mass behind it, kTailBits more
  int list_window, list_from, list_to; // bins whose tokens are listed
  unsigned listed;

  __device__ void ask(const Order& o) {
    if (threadIdx.x == 0) s.order = o;
    cluster_sync();
    serve(s, s, cluster, o, part, scale);
  }
  // Sums before each bin, from the bins' own.
  __device__ void add_up() {
    const int b = 2 * threadIdx.x;
    const uint64_t m0 = s.mass_before[b], m1 = s.mass_before[b + 1];
    const unsigned c0 = s.count_before[b], c1 = s.count_before[b + 1];
    uint64_t mb;
    unsigned cb;
    scan_before(s, m0 + m1, c0 + c1, &mb, &cb, &mass, &count);
    s.mass_before[b] = mb;
    s.mass_before[b + 1] = mb + m0;
    s.count_before[b] = cb;
    s.count_before[b + 1] = cb + c0;
    if (threadIdx.x == 0) {
      s.mass_before[kBins] = mass;
      s.count_before[kBins] = count;
    }
    __syncthreads();
  }
  // Bins hold sums of 30-bit weights; a mass is that at the octave's place.
  __device__ void to_masses() {
    for (int b = threadIdx.x; b < kBins; b += kThreads) s.mass_before[b] <<= kOctaves - 1 - b / kSub;
    __syncthreads();
  }
  __device__ void take_window(int w) {
    to_masses();
    add_up();
    tail = 0;
    for (int p = 0; p < static_cast<int>(cluster.num_blocks()); ++p) tail += s.tails[p];
    window = w;
  }
  __device__ void need_window(int w) {
    if (window == w) return;
    ask(Order{kOpBins, w, 0, 0, 0, 0, 0});
    take_window(w);
  }
  // The bin (or digit) with before[b] <= target < before[b + 1].
  template <typename V>
  __device__ int find(const V* before, V target) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int b = 2 * threadIdx.x + q;
      if (before[b] <= target && target < before[b + 1]) s.found = b;
    }
    __syncthreads();
    const int b = s.found;
    __syncthreads();
    return b;
  }

  // The token among the listed ones of a bin where the sum passes `target`: a count, or a sum of weights.
  __device__ uint64_t among_listed(int bin, bool by_count, uint64_t target, uint64_t* before, unsigned* own) {
    uint64_t key[kEach];
    unsigned w[kEach];
    bool in[kEach];
    uint64_t any = 0, all = ~uint64_t(0);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      const unsigned i = q * kThreads + threadIdx.x;
      in[q] = i < listed;
      key[q] = in[q] ? s.list[i] : 0;
      const float x = value_of(key[q]);
      float t;
      const int j = bin_of(x, scale, &t);
      in[q] = in[q] && j == bin;
      w[q] = in[q] ? weight_in(x, j, t, scale, s.middle) : 0;
      if (in[q]) {
        any |= key[q];
        all &= key[q];
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      any |= __shfl_xor_sync(~0u, any, d);
      all &= __shfl_xor_sync(~0u, all, d);
    }
    if (threadIdx.x % 32 == 0) {
      s.warp_mass[threadIdx.x / 32] = any;
      s.mass_before[threadIdx.x / 32] = all;  // (scratch here; saved by the caller)
    }
    __syncthreads();
    any = 0;
    all = ~uint64_t(0);
    for (int i = 0; i < kWarps; ++i) {
      any |= s.warp_mass[i];
      all &= s.mass_before[i];
    }
    __syncthreads();
    uint64_t differ = any ^ all;  // (one token: none)
    *before = 0;
    while (differ) {
      const int top = 63 - __clzll(static_cast<long long>(differ));
      const int shift = top >= kDigitBits - 1 ? top - (kDigitBits - 1) : 0;
      s.count[threadIdx.x] = s.low[threadIdx.x] = s.high[threadIdx.x] = 0;
      __syncthreads();
      int digit[kEach];
#pragma unroll
      for (int q = 0; q < kEach; ++q) {
        digit[q] = (1 << kDigitBits) - 1 - static_cast<int>((key[q] >> shift) & ((1 << kDigitBits) - 1));
        if (!in[q]) continue;
        atomicAdd(&s.count[digit[q]], 1u);
        atomicAdd(&s.low[digit[q]], w[q] & 0x7fffu);
        atomicAdd(&s.high[digit[q]], w[q] >> 15);
      }
      __syncthreads();
      const uint64_t m = s.low[threadIdx.x] + (static_cast<uint64_t>(s.high[threadIdx.x]) << 15);
      const unsigned c = s.count[threadIdx.x];
      uint64_t mb, ma;
      unsigned cb, ca;
      scan_before(s, m, c, &mb, &cb, &ma, &ca);
      const uint64_t b0 = by_count ? cb : mb, b1 = by_count ? cb + c : mb + m;
      if (b0 <= target && target < b1) {
        s.found = static_cast<int>(threadIdx.x);
        s.tails[0] = mb;
        s.tails[1] = b0;
      }
      __syncthreads();
      const int sel = s.found;
      *before += s.tails[0];
      target -= s.tails[1];
      const bool sole = s.count[sel] == 1;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kEach; ++q) in[q] = in[q] && digit[q] == sel;
      differ = sole || shift == 0 ? 0 : differ & ((uint64_t(1) << shift) - 1);
    }
#pragma unroll
    for (int q = 0; q < kEach; ++q)
      if (in[q]) {
        s.found_key = key[q];
        s.found = static_cast<int>(w[q]);
      }
    __syncthreads();
    const uint64_t k = s.found_key;
    *own = static_cast<unsigned>(s.found);
    __syncthreads();
    return k;
  }

  // The token of bin b of the window where the sum (relative to the bin's start) passes `target`.
  __device__ uint64_t in_bin(int b, bool by_count, uint64_t target, uint64_t* before, unsigned* own) {
    uint64_t mask = 0, value = 0, past = 0;
    unsigned held = s.count_before[b + 1] - s.count_before[b];
    if (!(list_window == window && b >= list_from && b < list_to)) {
      int from = b;
      if (s.count_before[b + 1] <= kCap) from = 0;
      else if (held > kCap) {
        // narrowed by digits over the cluster: the window's sums are made anew afterwards
        const int w = window;
        ask(Order{kOpBits, w, b, b + 1, 0, 0, 0});
        uint64_t any = 0, all = ~uint64_t(0);
        for (int p = 0; p < static_cast<int>(cluster.num_blocks()); ++p) {
          any |= s.ors[p];
          all &= s.ands[p];
        }
        int top = 64 - __clzll(static_cast<long long>(any ^ all));
        mask = ~((uint64_t(1) << top) - 1);
        value = all & mask;
        while (held > kCap) {
          const int shift = top > kDigitBits ? top - kDigitBits : 0;
          ask(Order{kOpDigits, w, b, b + 1, mask, value, shift});
          add_up();
          const int digit = by_count ? find(s.count_before, static_cast<unsigned>(target)) : find(s.mass_before, target);
          held = s.count_before[digit + 1] - s.count_before[digit];
          past += s.mass_before[digit];
          target -= by_count ? s.count_before[digit] : s.mass_before[digit];
          // (digits below bit `shift` are still open; the digit's own bits above `top` are the mask's)
          const uint64_t bits = static_cast<uint64_t>((1 << kDigitBits) - 1 - digit) << shift;
          const uint64_t open = (uint64_t(1) << shift) - 1;
          value = (value & mask) | (bits & ~mask);
          mask = ~open;
          value &= mask;
          top = shift;
          __syncthreads();
        }
        window = -1;
        if (threadIdx.x == 0) s.listed = 0;
        ask(Order{kOpGather, w, b, b + 1, mask, value, 0});
        list_window = -1;
        listed = min(s.listed, static_cast<unsigned>(kCap));
        const uint64_t key = among_listed(w * kBins + b, by_count, target, before, own);
        *before += past;
        return key;
      }
      if (threadIdx.x == 0) s.listed = 0;
      ask(Order{kOpGather, window, from, b + 1, 0, 0, 0});
      list_window = window;
      list_from = from;
      list_to = b + 1;
      listed = min(s.listed, static_cast<unsigned>(kCap));
    }
    // (the search by digits uses the first places of the bins' sums)
    uint64_t saved = 0;
    if (threadIdx.x < kWarps) saved = s.mass_before[threadIdx.x];
    __syncthreads();
    const uint64_t key = among_listed(window * kBins + b, by_count, target, before, own);
    if (threadIdx.x < kWarps) s.mass_before[threadIdx.x] = saved;
    __syncthreads();
    return key;
  }

  __device__ Crossing where(bool by_count, uint64_t target) {
    uint64_t done = 0;  // mass of the windows before, in the unit of window 0
    for (int w = 0; w < kWindows; ++w) {
      need_window(w);
      uint64_t t = by_count ? target : (target - done) << (kOctaves * w);
      const uint64_t all = by_count ? count : mass;
      const bool last = tail == 0;
      if (t >= all && last && !by_count && all) t = all - 1;  // (sums of different units, rounded: the last token)
      if (t < all) {
        const int b = by_count ? find(s.count_before, static_cast<unsigned>(t)) : find(s.mass_before, t);
        const uint64_t start = s.mass_before[b], first = by_count ? s.count_before[b] : start;
        const int up = kOctaves - 1 - b / kSub;
        uint64_t before;
        unsigned own;
        const uint64_t key = in_bin(b, by_count, by_count ? t - first : (t - first) >> up, &before, &own);
        return Crossing{true, key, done + ((start + ((before + own) << up)) >> (kOctaves * w))};
      }
      if (last) break;
      if (by_count) target -= count;
      done += mass >> (kOctaves * w);
      if (!by_count && target < done) target = done;
    }
    return Crossing{false, 0, 0};
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) token_kernel(const TokenDraw p, int slots) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kVec = 16 / sizeof(T);
  Shared& s = *reinterpret_cast<Shared*>(smem);
  T* data = reinterpret_cast<T*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
  const int64_t row = blockIdx.x / blocks;
  if (threadIdx.x < kSub) s.middle[threadIdx.x] = kMiddles.v[threadIdx.x];
  if (threadIdx.x == 0) s.found = 0;
  grid_dependency_wait();
  grid_launch_dependents();

  // the block's part into shared memory, with the row's maximum; slots start on a 16-byte boundary at or before the row
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) % kVec);
  Part<T> part{data, slots, rank * slots - lead};
  float most = -INFINITY;
  for (int at = threadIdx.x * kVec; at < slots; at += kThreads * kVec) {
    const int i = part.index0 + at;
    Vec<T, kVec> v;
    if (i >= 0 && i + kVec <= p.n) {
      v.set(ld_stream_v4(x + i));
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v.v[e] = i + e >= 0 && i + e < p.n ? to_f32(x[i + e]) : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) most = fmaxf(most, v.v[e]);
    v.store(data + at);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
  if (threadIdx.x % 32 == 0) s.warp_count[threadIdx.x / 32] = __float_as_uint(most);
  cluster_sync();  // (every block has started, too)
  if (threadIdx.x < blocks) {
    for (int w = 0; w < kWarps; ++w) most = fmaxf(most, __uint_as_float(s.warp_count[w]));
    cluster.map_shared_rank(&s, threadIdx.x)->maxes[rank] = most;
  }
  cluster_sync();
  most = s.maxes[0];
  for (int b = 1; b < blocks; ++b) most = fmaxf(most, s.maxes[b]);
  if (most == -INFINITY) {  // nothing that may be drawn (in every block alike)
    if (rank == 0 && threadIdx.x == 0) {
      p.tokens[row] = -1;
      p.logprobs[row] = -INFINITY;
    }
    return;
  }

  const float temperature = p.temperatures ? p.temperatures[row] : p.temperature;
  const float min_p = p.min_ps ? p.min_ps[row] : p.min_p;
  const bool greedy = !(temperature > 0.0f);
  Scale scale{most, -FLT_MAX, FLT_MAX, 0.0f};
  if (!greedy) {
    const double per = 1.4426950408889634 / static_cast<double>(temperature);
    if (per < FLT_MAX) {
      scale.hi = static_cast<float>(per);
      scale.lo = static_cast<float>(per - static_cast<double>(scale.hi));
    }
    if (min_p > 0.0f) {  // w >= min_p: x >= max + T ln(min_p)
      const double least = static_cast<double>(most) + static_cast<double>(temperature) * log(static_cast<double>(min_p));
      const float f = __double2float_ru(least);
      scale.least = fminf(fmaxf(f, -FLT_MAX), most);
    }
  } else {
    scale.least = most;
  }

  Shared& first = *cluster.map_shared_rank(&s, 0);
  serve(s, first, cluster, Order{kOpBins, 0, 0, 0, 0, 0, 0}, part, scale);
  if (rank != 0) {
    for (;;) {
      cluster_sync();
      const Order o = first.order;
      if (o.op == kOpDone) break;
      serve(s, first, cluster, o, part, scale);
    }
    cluster_sync();
    return;
  }
  Search<T> search{s, cluster, part, scale, 0, 0, 0, 0, -1, 0, 0, 0};
  search.take_window(0);
  uint64_t kept = search.mass + (search.tail >> kTailBits);
  const int top_k = greedy ? 1 : p.top_ks ? p.top_ks[row] : p.top_k;
  const float top_p = p.top_ps ? p.top_ps[row] : p.top_p;
  const float u = p.u[row];
  if (top_k > 0 && top_k < p.n) {
    const Crossing c = search.where(true, static_cast<uint64_t>(top_k - 1));
    if (c.found) kept = c.through;
  }
  if (top_p < 1.0f) {
    // the first prefix with a mass of at least top_p of it: the sum before its last token is below that
    const double border = ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(kept));
    const uint64_t target = border < 1.0 ? 0 : static_cast<uint64_t>(border) - 1;
    const Crossing c = search.where(false, target < kept ? target : kept - 1);
    if (c.found && c.through < kept) kept = c.through;
  }
  const double drawn = (u > 0.0f ? static_cast<double>(u) : 0.0) * static_cast<double>(kept);
  const uint64_t target = drawn < static_cast<double>(kept) ? static_cast<uint64_t>(drawn) : kept;
  const Crossing c = search.where(false, target < kept ? target : kept - 1);
  if (threadIdx.x == 0) {
    p.tokens[row] = c.found ? index_of(c.key) : -1;
    const float x0 = value_of(c.key);
    const double z = greedy || x0 == most ? 0.0 : (static_cast<double>(x0) - static_cast<double>(most)) / static_cast<double>(temperature);
    const double share = static_cast<double>(kept) * 0x1p-45;  // (the largest weight is 2^45)
    p.logprobs[row] = fminf(static_cast<float>(z - log(share)), 0.0f);
    s.order = Order{kOpDone, 0, 0, 0, 0, 0, 0};
  }
  cluster_sync();
  cluster_sync();
}

}  // namespace

template <typename T>
static cudaError_t launch(const TokenDraw& p, cudaStream_t st) {
  constexpr int64_t kVec = 16 / sizeof(T);
  // blocks a row: 64 KB of it each, so that two blocks share an SM and one loads while the other searches; more where rows
  // are few, down to 4096 tokens each
  const int64_t len = p.n + kVec;
  int blocks = 1;
  while (blocks < 8 && (len * static_cast<int64_t>(sizeof(T)) > blocks * 65536 || (p.rows * blocks * 2 <= ops_sm_count() && len > blocks * 4096)))
    blocks *= 2;
  const int64_t slots = ((len + blocks - 1) / blocks + kVec - 1) / kVec * kVec;
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + static_cast<size_t>(slots) * sizeof(T);
  cudaError_t e = cudaFuncSetAttribute(token_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  if (p.rows * blocks > INT32_MAX) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows * blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_kernel<T>, p, static_cast<int>(slots));
}

cudaError_t launch_tokens(const TokenDraw& p, cudaStream_t st) {
  return p.dtype == kF32 ? launch<float>(p, st) : launch<__nv_bfloat16>(p, st);
}

}  // namespace tk

// Matrix products c = act(a b^T + bias) + residual on the tensor cores
// (tcgen05.mma, bf16 operands, f32 accumulators in tensor memory).
//
// A persistent grid of CTA pairs takes 256 x 256 tiles of c in turn, each pair
// sharing one product (cta_group::2: each CTA holds half of a's rows and half
// of b's).  In each CTA one thread brings the operands' slices into a ring of
// shared-memory stages by TMA (128-byte swizzle, zeros outside the matrices),
// one thread of the leading CTA issues the products from them, and eight warps
// read finished accumulators from tensor memory, apply bias, activation and
// residual in f32, round once and store.  Tensor memory holds two
// accumulators, so that a tile's results are written while the next tile is
// multiplied.
//
// The last tiles rarely fill the pairs evenly.  Where it pays, the stages of
// the tiles past the last whole wave (all of them when there is no whole wave)
// are dealt to the pairs in equal runs, whatever tile they fall in: a run that
// covers part of a tile's k leaves its f32 sums in scratch, and of the warps
// that do so for the same rows and columns the last one (by a ticket) adds the
// parts in order of k and writes the result.  Nothing waits for another run.
//
// F32 operands are taken apart into three bf16 parts each, every part what the
// ones before it left, rounded to nearest (8 + 8 + 8 bits and two signs: nothing
// is left), and the six products of parts whose orders add up to at most two
// are summed, the smallest first.  The dropped ones are at most 2^-24 of a
// product (parts of orders one and two are within 2^-8 and 2^-17 of a value's
// exponent) and of either sign; with parts that were cut off they had the
// product's sign and reached 2^-21.  So a stage is one of six times as many;
// results are f32.  An infinity would meet a zero part (NaN): where the split
// finds one, the product is made on the CUDA cores and this kernel does nothing.
// An operand with values whose third part bf16 cannot hold is split anew,
// scaled by a power of two that the results are freed of.
//
// A bf16 operand a whose values have a rest (the gradient of a smooth
// activation) is multiplied as two parts, a stage of k of both in turn: twice
// as many stages.  The rest's sign is its own, so an infinity in b would meet
// both signs, or a zero (NaN): where one is found, the leading part takes the
// rest's place too and the sums are halved.
//
// Every wait has a limit, after which the status word is set and the kernel
// winds up.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <mutex>

#include "ops_common.cuh"

namespace tk {
namespace {

constexpr int kDeepK = 64;             // k of one stage: 128 bytes of bf16
constexpr int kTileM = 128;            // rows of c in one CTA
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kStageBytesOut = 4096;   // staging of one epilogue warp: 32 rows x 128 bytes

// The tensor cores' sums are cut off, not rounded, so that a long sum drifts
// (K = 4096 in one accumulator: 4.5e-6 of the result, and in proportion to K).
// After a round of k the sums therefore go to f32 registers, where they are
// added to those before (rounded); the last round's accumulator takes their
// total.  Rounds are eight stages of k (all six products of them) for f32,
// which leaves 5e-7, and 32 for bf16 (16 where each has two products), which
// leaves 2.3e-6 whatever K, what an f32 sum of some 10^4 terms has.  Each
// reading of an accumulator holds the products up by some 0.3 us (bf16 8192 x
// 8192 x 8192: one sum 588 us, rounds of 32 stages 619, of 16 631, of 8 655).
// (TERMS: the products of parts that make one of values.)
constexpr int kTermsF32 = 6, kTermsRest = 2;
template <int TERMS>
constexpr int kRoundDepthOf = TERMS == kTermsF32 ? 8 : TERMS == kTermsRest ? 16 : 32;  // stages of k in a round
constexpr int kTileN = 256;            // columns of c in a pair's tile (and of tensor memory in an accumulator)
constexpr int kPairM = 2 * kTileM;     // its rows
constexpr int kRowsB = kTileN / 2;     // rows of b that one CTA brings in
constexpr int kBytesA = kTileM * kDeepK * 2, kBytesB = kRowsB * kDeepK * 2;
constexpr int kStage = kBytesA + kBytesB;
constexpr int kStages = 6;
constexpr int kOffStaging = kStages * kStage;
constexpr int kOffBias = kOffStaging + kEpiWarps * kStageBytesOut;
constexpr int kOffBars = kOffBias + 2 * kTileN * 4;
constexpr int kSmem = kOffBars + (2 * kStages + 4) * 8 + 16;
static_assert(kSmem <= 232448, "shared memory of one CTA");

// How the stages of all tiles are dealt to `pairs` pairs: `waves` whole tiles
// to each, then the stages of the remaining `shared_tiles` in equal runs.
struct Deal {
  int tiles_m, tiles_n;
  int k_blocks;       // stages of a tile
  int depth;          // those of one product of parts (k_blocks where values have one part)
  int pairs;
  int waves;
  int shared_tiles;   // 0: every pair's tiles are whole (the last wave may be short)
  int run, longer;    // stages of a run; the first `longer` pairs' runs have one more
  __device__ __forceinline__ int run_start(int pair) const { return pair * run + min(pair, longer); }
  // The pair whose run holds a stage (counted over the shared tiles).
  __device__ __forceinline__ int run_of(int stage) const {
    const int head = longer * (run + 1);
    return stage < head ? stage / (run + 1) : longer + (stage - head) / run;
  }
};

struct MmaParams {
  CUtensorMap a, b, c, pre;
  int64_t m, n;
  Deal deal;
  bool a_k, b_k;           // operand order: k contiguous
  uint32_t idesc;
  const void* bias;        // nullable
  const void* residual;    // nullable
  int64_t ldr;
  int act;
  bool tma_c, tma_pre;     // stores by TMA (else by plain stores)
  void* c_ptr;
  int64_t ldc;
  void* pre_ptr;           // nullable
  int64_t ldp;
  float* part;             // sums of parts of k: 2 slots a pair, each kPairM x kTileN
  unsigned* ticket;        // 2 kEpiWarps a shared tile, zero between launches
  const int* marks;        // of operands in parts, as `call` left them
  int call;
  int* status;
};

// ---- PTX --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// Arrivals on a barrier of any CTA of the cluster (bar: its shared::cluster address).
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Waits for phase `parity`, at most kWaitLimitNs; false when it gave up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (;;) {
    // (the timer is slow to read: only once in many tries)
    for (int i = 0; i < 256; ++i)
      if (bar_try(bar, parity)) return true;
    const uint64_t t = globaltimer_ns();
    if (!t0) t0 = t;
    if (t - t0 > kWaitLimitNs) return false;
  }
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
               "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
               ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
// Arrives on `bar` (at the same place in both CTAs) when the products issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(bar), "h"(uint16_t(3)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of the warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The same of 8 columns, and back.
__device__ __forceinline__ void tmem_load8(uint32_t addr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const float* v) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Shared-memory descriptor of an operand slice in the 128-byte swizzle: rows
// (k contiguous) or columns of 8 x 128 bytes 1024 bytes apart; with the rows
// contiguous, the groups of 64 rows `lead` bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t(addr >> 4) & 0x3fff) | (uint64_t(lead >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// A pair's next piece of work: stages [kb0, kb1) of a tile.
struct Work {
  int m, n;
  int kb0, kb1;
  int slot;   // where its sums go when it covers only part of k; -1: a whole tile
  int shared; // the tile's number among the shared ones
};
// Tiles in strips of kStrip tile rows, down the strip first: pairs that run at
// the same time share rows of b and keep a strip of a in L2.
constexpr int kStrip = 16;
__device__ __forceinline__ void tile_at(const Deal& d, int t, int* m, int* n) {
  const int strip = t / (kStrip * d.tiles_n);
  const int first = strip * kStrip;
  const int tall = min(kStrip, d.tiles_m - first);
  const int in = t - strip * kStrip * d.tiles_n;
  *m = first + in % tall;
  *n = in / tall;
}
struct Worker {
  int pair, wave;
  int at, end;  // the pair's run of stages, counted over the shared tiles
  __device__ __forceinline__ Worker(const Deal& d, int pair_) : pair(pair_), wave(0) {
    at = d.shared_tiles ? d.run_start(pair) : 0;
    end = d.shared_tiles ? d.run_start(pair + 1) : 0;
  }
  __device__ __forceinline__ void leave() {
    wave = INT32_MAX;
    at = end;
  }
  __device__ __forceinline__ bool next(const Deal& d, Work* w) {
    const int64_t tile = int64_t(wave) * d.pairs + pair;
    if (wave < d.waves && tile < int64_t(d.tiles_m) * d.tiles_n) {
      ++wave;
      tile_at(d, static_cast<int>(tile), &w->m, &w->n);
      w->kb0 = 0;
      w->kb1 = d.k_blocks;
      w->slot = -1;
      return true;
    }
    if (at >= end) return false;
    const int t = at / d.k_blocks;
    w->kb0 = at - t * d.k_blocks;
    w->kb1 = min(d.k_blocks, w->kb0 + (end - at));
    // a run begins at most one tile in its middle (slot 2 pair) and leaves at most one tile from its start (2 pair + 1)
    w->slot = w->kb0 > 0 ? 2 * pair : w->kb1 < d.k_blocks ? 2 * pair + 1 : -1;
    w->shared = t;
    tile_at(d, d.waves * d.pairs + t, &w->m, &w->n);
    at += w->kb1 - w->kb0;
    return true;
  }
};

// ---- the epilogue's tile chunk: 32 rows x 128 bytes in a warp's staging ---------------
// 16-byte piece `q` (0..7) of row `row`, at its place in the 128-byte swizzle.
__device__ __forceinline__ uint32_t piece(uint32_t staging, int row, int q) {
  return staging + row * 128 + ((q ^ (row & 7)) << 4);
}

// Plain stores of the staged chunk, for results whose rows TMA cannot address.
template <typename T>
__device__ __forceinline__ void store_plain(uint32_t staging, T* dst, int64_t ld, int64_t row0, int64_t rows, int64_t col0,
                                            int64_t cols, int lane) {
  constexpr int kCols = 128 / sizeof(T);
#pragma unroll 4
  for (int r = 0; r < 32; ++r) {
    if (row0 + r >= rows) break;
#pragma unroll
    for (int e = 0; e < kCols / 32; ++e) {
      const int c = e * 32 + lane;
      const uint32_t addr = piece(staging, r, c * int(sizeof(T)) / 16) + (c * sizeof(T)) % 16;
      T v;
      if constexpr (sizeof(T) == 2) {
        uint16_t u;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(addr) : "memory");
        v = __ushort_as_bfloat16(u);
      } else {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
      }
      if (col0 + c < cols) dst[(row0 + r) * ld + col0 + c] = v;
    }
  }
}
// A chunk of the residual into staging, zeros outside it (any alignment, rows read in order).
template <typename T>
__device__ __forceinline__ void stage_residual(uint32_t staging, const T* src, int64_t ld, int64_t row0, int64_t rows,
                                               int64_t col0, int64_t cols, int lane) {
  constexpr int kEach = 4 / sizeof(T), kRows = 32 / kEach;  // loads of 32 values in flight
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += kRows) {
    T v[kRows][kEach];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int c = e * 32 + lane;
        v[r][e] = from_f32<T>(0.0f);
        if (row0 + r0 + r < rows && col0 + c < cols) v[r][e] = src[(row0 + r0 + r) * ld + col0 + c];
      }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int c = e * 32 + lane;
        const uint32_t addr = piece(staging, r0 + r, c * int(sizeof(T)) / 16) + (c * sizeof(T)) % 16;
        if constexpr (sizeof(T) == 2)
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(__bfloat16_as_ushort(v[r][e])) : "memory");
        else
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v[r][e]) : "memory");
      }
  }
}
// 32 values of the lane's row, rounded to T, into staging: half `h` of its 128 bytes (bf16), or all (f32).
template <typename T>
__device__ __forceinline__ void stage_values(uint32_t staging, int lane, int h, const float* v) {
  constexpr int kVec = 16 / sizeof(T), kPieces = 32 / kVec;
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    Vec<T, kVec> o;
#pragma unroll
    for (int i = 0; i < kVec; ++i) o.v[i] = v[q * kVec + i];
    const uint4 u = o.pack();
    st_shared16(piece(staging, lane, kPieces * h + q), u.x, u.y, u.z, u.w);
  }
}
template <typename T, int N>
__device__ __forceinline__ void apply_act(float* v, int act) {
  if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = relu(v[i]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value<T>(v[i], kActGelu);
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value<T>(v[i], kActSilu);
  }
}
__device__ __forceinline__ void add_bias32(float* v, const float* bias) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 t = reinterpret_cast<const float4*>(bias)[i];
    v[4 * i] += t.x;
    v[4 * i + 1] += t.y;
    v[4 * i + 2] += t.z;
    v[4 * i + 3] += t.w;
  }
}

__device__ __forceinline__ void scale32(float* v, float f) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] *= f;
}

// The pairs whose runs meet shared tile t, [first, first + parts).
__device__ __forceinline__ void runs_of_tile(const Deal& d, int t, int* first, int* parts) {
  *first = d.run_of(t * d.k_blocks);
  *parts = d.run_of(t * d.k_blocks + d.k_blocks - 1) + 1 - *first;
}
// The warp has read its accumulator (bar: the leading CTA's barrier counts both CTAs' warps).
__device__ __forceinline__ void free_accumulator(int lane, uint32_t bar) {
  fence_before();
  __syncwarp();
  if (lane == 0) bar_arrive(map_to_rank(bar, 0));
}

template <typename T, int TERMS>
__global__ void __cluster_dims__(2) __launch_bounds__(kThreads, 1) mma_kernel(const __grid_constant__ MmaParams p) {
  constexpr int kRoundDepth = kRoundDepthOf<TERMS>, kRoundStages = TERMS * kRoundDepth;
  const T* bias = static_cast<const T*>(p.bias);
  const T* residual = static_cast<const T*>(p.residual);
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_addr(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const uint32_t bars = base + kOffBars;
  auto full = [&](int s) { return bars + s * 8; };
  auto empty = [&](int s) { return bars + (kStages + s) * 8; };
  auto acc_full = [&](int b) { return bars + (2 * kStages + b) * 8; };
  auto acc_empty = [&](int b) { return bars + (2 * kStages + 2 + b) * 8; };
  const uint32_t tmem_word = bars + (2 * kStages + 4) * 8;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(full(s), 2);   // each CTA's loads
      bar_init(empty(s), 1);  // the products that read the stage
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(acc_full(b), 1);
      bar_init(acc_empty(b), 2 * kEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc(tmem_word, 2 * kTileN);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_word) : "memory");
  // what comes before this grid is not needed until here
  grid_dependency_wait();
  grid_launch_dependents();

  Worker worker(p.deal, blockIdx.x / 2);
  bool twice = false;   // the leading part in the rest's place too
  float undo = 1.0f;    // a power of two that the sums are multiplied by
  if constexpr (TERMS == kTermsF32) {
    const PartsPlan plan = parts_plan(p.marks, p.call);
    if (plan.cores) worker.leave();
    undo = (plan.scale_a ? kUnscale : 1.0f) * (plan.scale_b ? kUnscale : 1.0f);
  } else if constexpr (TERMS == kTermsRest) {
    twice = p.marks[kMarkOther] == p.call;
    if (twice) undo = 0.5f;
  }
  Work w;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {  // loads
      int stage = 0;
      uint32_t phase = 0;
      while (ok && worker.next(p.deal, &w)) {
        const int m0 = w.m * kPairM + static_cast<int>(rank) * kTileM;
        const int n0 = w.n * kTileN + static_cast<int>(rank) * kRowsB;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!(ok = bar_wait(empty(stage), phase ^ 1))) break;
          const uint32_t sa = base + stage * kStage, sb = sa + kBytesA;
          const uint32_t bar = map_to_rank(full(stage), 0);
          bar_expect(bar, kStage);
          int k0 = kb * kDeepK, part_a = 0, part_b = 0;
          if constexpr (TERMS == kTermsF32) {
            // a round's products of parts one after the other: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0)
            const int round = kb / kRoundStages, in = kb - round * kRoundStages;
            const int deep = min(kRoundDepth, p.deal.depth - round * kRoundDepth), term = in / deep;
            k0 = (round * kRoundDepth + in - term * deep) * kDeepK;
            part_a = 0x001102 >> (4 * term) & 3;
            part_b = 0x010120 >> (4 * term) & 3;
          } else if constexpr (TERMS == kTermsRest) {
            // rest and leading part of a stage of k in turn: b's slice is then in L2 (one after the other over a round,
            // 2000 x 4096 x 16384 took 871 us instead of 757)
            k0 = (kb >> 1) * kDeepK;
            part_a = ~kb & 1;
            if (twice) part_a = 0;
          }
          if (p.a_k) {
            tma_load(sa, &p.a, k0, m0, part_a, bar);
          } else {
            tma_load(sa, &p.a, m0, k0, part_a, bar);
            tma_load(sa + 8192, &p.a, m0 + 64, k0, part_a, bar);
          }
          if (p.b_k) {
            tma_load(sb, &p.b, k0, n0, part_b, bar);
          } else {
            tma_load(sb, &p.b, n0, k0, part_b, bar);
            tma_load(sb + 8192, &p.b, n0 + 64, k0, part_b, bar);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // every stage has been read before this CTA ends
      for (int s = 0; s < kStages && ok; ++s) {
        ok = bar_wait(empty(stage), phase ^ 1);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {  // products
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      const uint32_t step_a = (p.a_k ? 32 : 2048) >> 4, step_b = (p.b_k ? 32 : 2048) >> 4;
      while (ok && worker.next(p.deal, &w)) {
        if (!(ok = bar_wait(acc_empty(buf), acc_phase ^ 1))) break;
        fence_after();
        uint32_t d = tmem + buf * kTileN;
        bool fresh = true;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (kb != w.kb0 && kb % kRoundStages == 0) {  // the round's sums go out, the next begins
            mma_commit(acc_full(buf));
            buf ^= 1;
            if (buf == 0) acc_phase ^= 1;
            if (!(ok = bar_wait(acc_empty(buf), acc_phase ^ 1))) break;
            fence_after();
            d = tmem + buf * kTileN;
            fresh = true;
          }
          if (!(ok = bar_wait(full(stage), phase))) break;
          fence_after();
          const uint32_t sa = base + stage * kStage, sb = sa + kBytesA;
          const uint64_t da = operand_desc(sa, 8192), db = operand_desc(sb, 8192);
#pragma unroll
          for (int i = 0; i < kDeepK / 16; ++i)
            mma(d, da + i * step_a, db + i * step_b, p.idesc, !fresh || i > 0);
          fresh = false;
          mma_commit(empty(stage));
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        mma_commit(acc_full(buf));
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1;
      }
    }
  } else if (warp >= 4) {  // results
    const int e = warp - 4, quad = e % 4, half = e / 4;
    const uint32_t staging = base + kOffStaging + e * kStageBytesOut;
    float* bias_smem = reinterpret_cast<float*>(smem + kOffBias);
    constexpr int kChunk = 128 / sizeof(T), kHalf = kTileN / 2;  // columns of the staging's 128 bytes
    int buf = 0, bias_buf = 0;
    uint32_t acc_phase = 0;
    for (; worker.next(p.deal, &w); bias_buf ^= 1) {
      const int64_t row0 = int64_t(w.m) * kPairM + rank * kTileM + quad * 32;
      const int64_t n0 = int64_t(w.n) * kTileN;
      if (bias) {
        for (int i = threadIdx.x - 128; i < kTileN; i += 32 * kEpiWarps)
          bias_smem[bias_buf * kTileN + i] = n0 + i < p.n ? to_f32(bias[n0 + i]) : 0.0f;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
      }
      const bool lies = row0 < p.m && n0 + half * kHalf < p.n;  // else nothing of the warp's part lies in c
      // a warp's part of a slot: four columns of each of its 32 rows together
      const int64_t region = (int64_t(rank) * kEpiWarps + e) * (32 * kHalf) + lane * 4;
      const uint32_t quad_at = half * kHalf + (uint32_t(quad * 32) << 16);
      // rounds before the last: their sums in registers (more than 8 columns on their way at a time would spill)
      float sum[kHalf] = {};
      bool held = false;
      for (int kb = (w.kb0 / kRoundStages + 1) * kRoundStages; kb < w.kb1; kb += kRoundStages) {
        if (ok) ok = __all_sync(~0u, bar_wait(acc_full(buf), acc_phase));
        fence_after();
        if (lies) {
#pragma unroll
          for (int c = 0; c < kHalf; c += 8) {
            float v[8];
            tmem_load8(tmem + buf * kTileN + quad_at + c, v);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[c + i] += v[i];
          }
        }
        free_accumulator(lane, acc_empty(buf));
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1;
        held = true;
      }
      // (a warp that gave up goes on without waiting, so that the others' barriers are still met)
      if (ok) ok = __all_sync(~0u, bar_wait(acc_full(buf), acc_phase));
      fence_after();
      const uint32_t acc = tmem + buf * kTileN + quad_at;
      if (!lies) {
        free_accumulator(lane, acc_empty(buf));
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1;
        continue;
      }
      if (held) {  // the accumulator takes the total
#pragma unroll
        for (int c = 0; c < kHalf; c += 8) {
          float v[8];
          tmem_load8(acc + c, v);
          tmem_wait_load();
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += sum[c + i];
          tmem_store8(acc + c, v);
        }
        tmem_wait_store();
      }
      int first = 0, parts = 0;  // pairs whose runs make up a shared tile
      if (w.slot >= 0) {
        float4* own = reinterpret_cast<float4*>(p.part + int64_t(w.slot) * (kPairM * kTileN) + region);
#pragma unroll 1
        for (int c0 = 0; c0 < kHalf; c0 += 32) {
          float v[32];
          tmem_load32(acc + c0, v);
          tmem_wait_load();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(own + c0 / 4 * 32 + i * 32, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        }
        free_accumulator(lane, acc_empty(buf));
        __threadfence();
        runs_of_tile(p.deal, w.shared, &first, &parts);
        __syncwarp();
        unsigned seen = 0;  // (counts up to parts - 1 and then back to 0 for the next launch)
        if (lane == 0) seen = atomicInc(&p.ticket[(w.shared * 2 + static_cast<int>(rank)) * kEpiWarps + e], parts - 1);
        seen = __shfl_sync(~0u, seen, 0);
        __threadfence();
        if (static_cast<int>(seen) != parts - 1) first = -1;
      }
      const float* bias_own = bias_smem + bias_buf * kTileN + half * kHalf;
      // 32 columns' sums (and the bias): from the accumulator, or from the parts, two parts' loads in flight
      auto fetch = [&](int c, float* v) {
        if (w.slot < 0) {
          tmem_load32(acc + c, v);
          tmem_wait_load();
        } else {
          const int k0 = w.shared * p.deal.k_blocks;
          auto part_of = [&](int pair) {
            const int slot = 2 * pair + (p.deal.run_start(pair) > k0 ? 0 : 1);
            return reinterpret_cast<const float4*>(p.part + int64_t(slot) * (kPairM * kTileN) + region) + c / 4 * 32;
          };
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll 1
          for (int o = 0; o < parts; o += 2) {
            const bool two = o + 1 < parts;
            const float4* s0 = part_of(first + o);
            const float4* s1 = part_of(first + o + (two ? 1 : 0));
            float4 t0[8], t1[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              t0[i] = __ldcg(s0 + i * 32);
              t1[i] = __ldcg(s1 + i * 32);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a[4] = {t0[i].x, t0[i].y, t0[i].z, t0[i].w}, b[4] = {t1[i].x, t1[i].y, t1[i].z, t1[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) v[4 * i + j] = (v[4 * i + j] + a[j]) + (two ? b[j] : 0.0f);
            }
          }
        }
        if (undo != 1.0f) scale32(v, undo);
        if (bias) add_bias32(v, bias_own + c);
      };
      if (sizeof(T) == 2 && w.slot < 0 && !p.pre_ptr && !residual) {
        // the usual case
        constexpr int kSteps = kChunk / 32;  // of a staged chunk
        auto finish = [&](int s, float* z) {
          if (s % kSteps == 0) {
            if (lane == 0) store_wait_read();  // the staging's last store has been read
            __syncwarp();
          }
          stage_values<T>(staging, lane, s % kSteps, z);
          if (s % kSteps == kSteps - 1) {
            const int64_t col0 = n0 + half * kHalf + (s / kSteps) * kChunk;
            fence_proxy_async_smem();
            __syncwarp();
            if (p.tma_c) {
              if (lane == 0 && col0 < p.n) {
                tma_store(&p.c, static_cast<int>(col0), static_cast<int>(row0), 0, staging);
                store_commit();
              }
            } else {
              store_plain(staging, static_cast<T*>(p.c_ptr), p.ldc, row0, p.m, col0, p.n, lane);
              __syncwarp();
            }
          }
        };
        if (p.act != kActGelu) {
          // 32 columns on their way from tensor memory while the 32 before them are finished
          float v[2][32];
          tmem_load32(acc, v[0]);
#pragma unroll
          for (int s = 0; s < kHalf / 32; ++s) {
            tmem_wait_load();
            if (s + 1 < kHalf / 32) tmem_load32(acc + 32 * (s + 1), v[(s + 1) & 1]);
            else free_accumulator(lane, acc_empty(buf));
            float* z = v[s & 1];
            if (undo != 1.0f) scale32(z, undo);
            if (bias) add_bias32(z, bias_own + 32 * s);
            if (p.act == kActRelu) apply_act<T, 32>(z, kActRelu);
            else if (p.act == kActSilu) apply_act<T, 32>(z, kActSilu);
            finish(s, z);
          }
        } else {
          // one copy of gelu's code (four, unrolled as above, took 348 us where this takes 299: they do not fit the
          // instruction cache)
#pragma unroll 1
          for (int s = 0; s < kHalf / 32; ++s) {
            float z[32];
            tmem_load32(acc + 32 * s, z);
            tmem_wait_load();
            if (s + 1 == kHalf / 32) free_accumulator(lane, acc_empty(buf));
            if (undo != 1.0f) scale32(z, undo);
            if (bias) add_bias32(z, bias_own + 32 * s);
            apply_act<T, 32>(z, kActGelu);
            finish(s, z);
          }
        }
        first = -1;
      }
#pragma unroll 1
      for (int c0 = 0; c0 < kHalf && first >= 0; c0 += kChunk) {
        const int64_t col0 = n0 + half * kHalf + c0;
        const bool inside = col0 < p.n && row0 < p.m;
        if (p.pre_ptr) {
          if (lane == 0) store_wait_read();  // the staging's last store has been read
          __syncwarp();
#pragma unroll 1
          for (int h = 0; h < kChunk / 32; ++h) {
            float v[32];
            fetch(c0 + 32 * h, v);
            stage_values<T>(staging, lane, h, v);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (p.tma_pre) {
            if (lane == 0 && inside) {
              tma_store(&p.pre, static_cast<int>(col0), static_cast<int>(row0), 0, staging);
              store_commit();
            }
          } else {
            store_plain(staging, static_cast<T*>(p.pre_ptr), p.ldp, row0, p.m, col0, p.n, lane);
          }
        }
        if (lane == 0) store_wait_read();
        __syncwarp();
        if (residual) {
          stage_residual(staging, residual, p.ldr, row0, p.m, col0, p.n, lane);
          __syncwarp();
        }
#pragma unroll 1
        for (int h = 0; h < kChunk / 32; ++h) {
          float v[32];
          fetch(c0 + 32 * h, v);
          if (w.slot < 0 && c0 + 32 * h + 32 == kHalf) free_accumulator(lane, acc_empty(buf));
          apply_act<T, 32>(v, p.act);
          if (residual) {
            constexpr int kVec = 16 / sizeof(T), kPieces = 32 / kVec;
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
              Vec<T, kVec> r;
              r.set(ld_shared16(piece(staging, lane, kPieces * h + q)));
#pragma unroll
              for (int i = 0; i < kVec; ++i) v[q * kVec + i] += r.v[i];
            }
          }
          stage_values<T>(staging, lane, h, v);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (p.tma_c) {
          if (lane == 0 && inside) {
            tma_store(&p.c, static_cast<int>(col0), static_cast<int>(row0), 0, staging);
            store_commit();
          }
        } else {
          store_plain(staging, static_cast<T*>(p.c_ptr), p.ldc, row0, p.m, col0, p.n, lane);
        }
      }
      buf ^= 1;
      if (buf == 0) acc_phase ^= 1;
    }
    if (lane == 0) store_wait_all();
  }
  if (!ok && p.status) *p.status = kDevTimeout;
  __syncwarp();
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  if (warp == 2) tmem_free(tmem, 2 * kTileN);
}

// Copies an operand whose rows TMA cannot address to rows of `ld` values (a multiple of 8).
__global__ void __launch_bounds__(256) align_rows_kernel(const __nv_bfloat16* src, int64_t lds, int64_t rows, int64_t cols,
                                                         __nv_bfloat16* dst, int64_t ld) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t per = (cols + 1023) / 1024;
  const int64_t r = blockIdx.x / per, c0 = (blockIdx.x % per) * 1024 + threadIdx.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t c = c0 + e * 256;
    if (r < rows && c < cols) dst[r * ld + c] = src[r * lds + c];
  }
}

// The three bf16 parts of both f32 operands, `plane` values apart, rows of `ld`
// values.  A part is what the parts before it left, rounded to bf16, and the
// three hold all 24 bits of a value of kSmall or more.
struct Split {
  const float* src;
  int64_t lds, rows, cols;
  __nv_bfloat16* dst;
  int64_t ld, plane;
  unsigned blocks;
};
constexpr int kSplitEach = 4;  // values of a thread, next to each other
// The values from place `at` on, times `scale`; *most and *least: the largest magnitude, and the smallest but zero (NaN
// counts as infinity).
__device__ __forceinline__ void split_values(const Split& s, int64_t at, float scale, float* most, float* least) {
  const int64_t per = (s.cols + kSplitEach - 1) / kSplitEach, r = at / per, c = (at - r * per) * kSplitEach;
  const float* src = s.src + r * s.lds + c;
  float v[kSplitEach];
#pragma unroll
  for (int e = 0; e < kSplitEach; ++e) v[e] = c + e < s.cols ? src[e] : 0.0f;
#pragma unroll
  for (int e = 0; e < kSplitEach; ++e) {
    const float m = fabsf(v[e]);
    *most = m <= *most ? *most : m < INFINITY ? m : INFINITY;
    if (m > 0.0f) *least = fminf(*least, m);
    v[e] *= scale;
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    uint32_t two[kSplitEach / 2];
#pragma unroll
    for (int e = 0; e < kSplitEach; e += 2) {
      const __nv_bfloat162 top = __floats2bfloat162_rn(v[e], v[e + 1]);
      two[e / 2] = *reinterpret_cast<const uint32_t*>(&top);
      v[e] -= __uint_as_float(two[e / 2] << 16);
      v[e + 1] -= __uint_as_float(two[e / 2] & 0xffff0000u);
    }
    // (rows of the parts hold a multiple of 8 values: the last store may go past cols, not past the row)
    *reinterpret_cast<uint2*>(s.dst + q * s.plane + r * s.ld + c) = make_uint2(two[0], two[1]);
  }
}
__device__ __forceinline__ int64_t split_places(const Split& s) { return s.rows * ((s.cols + kSplitEach - 1) / kSplitEach); }

__global__ void __launch_bounds__(256) split_rows_kernel(const Split a, const Split b, int* marks, int call) {
  grid_dependency_wait();
  grid_launch_dependents();
  const bool second = blockIdx.x >= a.blocks;
  const Split& s = second ? b : a;
  const int64_t at = int64_t(blockIdx.x - (second ? a.blocks : 0)) * 256 + threadIdx.x;
  if (at >= split_places(s)) return;
  float most = 0.0f, least = INFINITY;
  split_values(s, at, 1.0f, &most, &least);
  if (!(most < 0x1.ffp127f)) marks[kMarkOther] = call;  // (what rounds to bf16's infinity included)
  if (most >= kLarge) marks[kMarkLarge] = call;
  if (least < kSmall) marks[second ? kMarkSmallB : kMarkSmallA] = call;
}
// The same again, scaled, for an operand that is marked so (a few blocks an SM: nothing, mostly).
__global__ void __launch_bounds__(256) split_scaled_kernel(const Split a, const Split b, const int* marks, int call) {
  grid_dependency_wait();
  grid_launch_dependents();
  const PartsPlan plan = parts_plan(marks, call);
  float most = 0.0f, least = 0.0f;
  const int64_t first = int64_t(blockIdx.x) * 256 + threadIdx.x, step = int64_t(gridDim.x) * 256;
  if (plan.scale_a)
    for (int64_t at = first; at < split_places(a); at += step) split_values(a, at, kScale, &most, &least);
  if (plan.scale_b)
    for (int64_t at = first; at < split_places(b); at += step) split_values(b, at, kScale, &most, &least);
}

// kMarkOther becomes `call` when a value of a bf16 matrix is not finite; a thread looks at eight values of a row.
__global__ void __launch_bounds__(256) mark_other_kernel(const __nv_bfloat16* p, int64_t ld, int64_t rows, int64_t cols, int* marks,
                                                         int call) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t per = (cols + 7) / 8, at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (at >= rows * per) return;
  const int64_t r = at / per, c = (at - r * per) * 8;
  const __nv_bfloat16* q = p + r * ld + c;
  bool finite = true;
  if (c + 8 <= cols && reinterpret_cast<uintptr_t>(q) % 16 == 0) {
    Raw<__nv_bfloat16, 8> v;
    v.load_nc(q);
    const uint32_t w[4] = {v.u.x, v.u.y, v.u.z, v.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) finite = finite && !__vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u);
  } else {
    for (int i = 0; i < 8 && c + i < cols; ++i) finite = finite && fabsf(to_f32(q[i])) < INFINITY;
  }
  if (!finite) marks[kMarkOther] = call;
}

// ---- host ------------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// A matrix of rows x cols values, rows ld apart, `planes` of them `plane` rows apart; boxes of box_cols x box_rows.
bool encode(CUtensorMap* map, bool f32, const void* p, int64_t cols, int64_t rows, int64_t ld, int64_t planes, int64_t plane,
            int box_cols, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const int size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(ld) * size, cuuint64_t(plane) * ld * size};
  const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr double kStageUs = 0.30, kJoinUs = 11.0;  // a stage of a tile, and the way of its parts, as timed

bool tma_rows(const void* p, int64_t ld, int size) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0; }

struct MmaPlan {
  Deal deal;
  __nv_bfloat16* copy_a;
  __nv_bfloat16* copy_b;
  int64_t ld_a, ld_b;  // of the copies, or of the operands where they serve as they are
  float* part;
};

int64_t operand_rows(const Operand& o, int64_t i, int64_t k) { return o.k_inner ? i : k; }
int64_t operand_cols(const Operand& o, int64_t i, int64_t k) { return o.k_inner ? k : i; }

// False when there are more tiles than a launch counts.
bool plan_mma(const Product& g, Scratch& sc, MmaPlan* q) {
  *q = MmaPlan{};
  Deal& d = q->deal;
  const int64_t tm = (g.m + kPairM - 1) / kPairM, tn = (g.n + kTileN - 1) / kTileN;
  if (tm > INT32_MAX / 4 / tn) return false;
  const int64_t tiles = tm * tn;
  d.tiles_m = static_cast<int>(tm);
  d.tiles_n = static_cast<int>(tn);
  const bool f32 = g.dtype == kF32;
  d.depth = static_cast<int>((g.k + kDeepK - 1) / kDeepK);
  if ((f32 || g.a.rest) && d.depth > INT32_MAX / kTermsF32) return false;
  d.k_blocks = (f32 ? kTermsF32 : g.a.rest ? kTermsRest : 1) * d.depth;
  const int slots = ops_sm_count() / 2 > 0 ? ops_sm_count() / 2 : 1;
  d.pairs = static_cast<int>(tiles < slots ? tiles : slots);
  d.waves = static_cast<int>((tiles + d.pairs - 1) / d.pairs);
  d.shared_tiles = 0;
  // Equal runs pay when the stages they save outweigh the parts' way through scratch.  Measured (one sum a tile): 4096 x 12288 x 512
  // (32 tiles of 192 stages) 60.7 -> 45.4 us, 12288 x 4096 x 512 (96 of 64) 48.0 -> 46.6; 300 x 4096 x 1000 (8 of 64)
  // 23.9 -> 25.1, 4096 x 1024 x 8192 (512 of 16) 44.5 -> 53.4, 2000 x 16384 x 4096 (128 of 256, where all SMs at once
  // draw the power limit) 158 -> 179.
  int pairs = 0;
  int64_t rest_waves = 0;
  if (tiles < slots) {
    // fewer tiles than pairs: as many pairs a tile as make the shortest run and its parts' way (a stage takes 0.17 us
    // where few SMs work, 0.30 where all do)
    auto stage_us = [&](double busy) { return 0.17 + 0.13 * busy / slots; };
    double best = d.k_blocks * stage_us(static_cast<double>(tiles));
    for (int64_t p = 2 * tiles; p < slots + tiles; p += tiles) {
      const int64_t used = p < slots ? p : slots;
      const double run = static_cast<double>(tiles) * d.k_blocks / used;
      const double t = run * stage_us(static_cast<double>(used)) + kJoinUs + 0.8 * used / tiles;
      if (run >= 2 && t < best) {
        best = t;
        pairs = static_cast<int>(used);
      }
    }
  } else if (tiles % slots != 0) {
    // the tiles past the last whole wave but one
    rest_waves = tiles / slots - 1;
    const int64_t shared = tiles - rest_waves * slots;
    const double even = static_cast<double>(shared) * d.k_blocks / slots;
    const double join = kJoinUs + 0.5 * slots / shared + 0.1 * static_cast<double>(tiles) * d.k_blocks / slots;
    if ((2 * d.k_blocks - even) * kStageUs > join) pairs = slots;
  }
  const int64_t shared = tiles - rest_waves * slots;
  if (pairs && shared * d.k_blocks <= INT32_MAX && shared * 2 * kEpiWarps <= kOpsWords - 64) {
    d.pairs = pairs;
    d.waves = static_cast<int>(rest_waves);
    d.shared_tiles = static_cast<int>(shared);
    d.run = static_cast<int>(shared * d.k_blocks / pairs);
    d.longer = static_cast<int>(shared * d.k_blocks % pairs);
  }
  if (d.shared_tiles) q->part = sc.take<float>(int64_t(2) * d.pairs * kPairM * kTileN);
  q->ld_a = g.a.ld;
  q->ld_b = g.b.ld;
  if (f32 || !tma_rows(g.a.p, g.a.ld, 2)) {
    q->ld_a = (operand_cols(g.a, g.m, g.k) + 7) / 8 * 8;
    q->copy_a = sc.take<__nv_bfloat16>((f32 ? 3 : 1) * q->ld_a * operand_rows(g.a, g.m, g.k));
  }
  if (f32 || !tma_rows(g.b.p, g.b.ld, 2)) {
    q->ld_b = (operand_cols(g.b, g.n, g.k) + 7) / 8 * 8;
    q->copy_b = sc.take<__nv_bfloat16>((f32 ? 3 : 1) * q->ld_b * operand_rows(g.b, g.n, g.k));
  }
  return true;
}

cudaError_t align_rows(const Operand& o, int64_t i, int64_t k, __nv_bfloat16* dst, int64_t ld, cudaStream_t st) {
  const int64_t rows = operand_rows(o, i, k), cols = operand_cols(o, i, k);
  const int64_t blocks = rows * ((cols + 1023) / 1024);
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  return launch_after(align_rows_kernel, static_cast<unsigned>(blocks), 256, 0, st, static_cast<const __nv_bfloat16*>(o.p), o.ld,
                      rows, cols, dst, ld);
}
bool split_of(const Operand& o, int64_t i, int64_t k, __nv_bfloat16* dst, int64_t ld, Split* s) {
  const int64_t rows = operand_rows(o, i, k), cols = operand_cols(o, i, k);
  const int64_t blocks = (rows * ((cols + kSplitEach - 1) / kSplitEach) + 255) / 256;
  if (blocks > INT32_MAX / 2) return false;
  *s = Split{static_cast<const float*>(o.p), o.ld, rows, cols, dst, ld, rows * ld, static_cast<unsigned>(blocks)};
  return true;
}

cudaError_t mark_other(const Operand& o, int64_t i, int64_t k, int* marks, int call, cudaStream_t st) {
  const int64_t rows = operand_rows(o, i, k), cols = operand_cols(o, i, k);
  const int64_t blocks = (rows * ((cols + 7) / 8) + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  return launch_after(mark_other_kernel, static_cast<unsigned>(blocks), 256, 0, st, static_cast<const __nv_bfloat16*>(o.p), o.ld,
                      rows, cols, marks, call);
}

template <typename T, int TERMS>
cudaError_t launch_mma_t(const MmaParams& p, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(mma_kernel<T, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(mma_kernel<T, TERMS>, static_cast<unsigned>(2 * p.deal.pairs), kThreads, kSmem, st, p);
}

}  // namespace

size_t mma_scratch_bytes(const Product& g) {
  Scratch sc;
  MmaPlan q;
  plan_mma(g, sc, &q);
  return sc.used();
}

cudaError_t launch_mma(const Product& g, Scratch& sc, const Words& words, int call, cudaStream_t st) {
  MmaPlan q;
  if (!plan_mma(g, sc, &q)) return cudaErrorNotSupported;
  const bool f32 = g.dtype == kF32;
  int* marks = words.at + kOpsMarks;
  cudaError_t e = cudaSuccess;
  if (f32) {
    Split a, b;
    if (!split_of(g.a, g.m, g.k, q.copy_a, q.ld_a, &a) || !split_of(g.b, g.n, g.k, q.copy_b, q.ld_b, &b)) return cudaErrorNotSupported;
    e = launch_after(split_rows_kernel, a.blocks + b.blocks, 256, 0, st, a, b, marks, call);
    const unsigned few = 4 * static_cast<unsigned>(ops_sm_count()), most = a.blocks > b.blocks ? a.blocks : b.blocks;
    if (e == cudaSuccess)
      e = launch_after(split_scaled_kernel, most < few ? most : few, 256, 0, st, a, b, static_cast<const int*>(marks), call);
  } else {
    if (q.copy_a) e = align_rows(g.a, g.m, g.k, q.copy_a, q.ld_a, st);
    if (e == cudaSuccess && q.copy_b) e = align_rows(g.b, g.n, g.k, q.copy_b, q.ld_b, st);
    if (e == cudaSuccess && g.a.rest) e = mark_other(g.b, g.n, g.k, marks, call, st);
  }
  if (e == cudaSuccess && f32) e = launch_simt(g, marks, call, st);
  if (e != cudaSuccess) return e;
  MmaParams p{};
  p.m = g.m;
  p.n = g.n;
  p.deal = q.deal;
  p.a_k = g.a.k_inner;
  p.b_k = g.b.k_inner;
  // f32 accumulators, bf16 operands, their order, and the product's size
  p.idesc = (1u << 4) | (1u << 7) | (1u << 10) | (p.a_k ? 0u : 1u << 15) | (p.b_k ? 0u : 1u << 16) |
            (static_cast<uint32_t>(kTileN / 8) << 17) | (static_cast<uint32_t>(kPairM / 16) << 24);
  const void* a = q.copy_a ? q.copy_a : g.a.p;
  const void* b = q.copy_b ? q.copy_b : g.b.p;
  const int64_t ra = operand_rows(g.a, g.m, g.k), rb = operand_rows(g.b, g.n, g.k);
  // (the parts of a lie ra rows apart, the rest of bf16 values too)
  if (g.a.rest && (q.copy_a || g.a.rest != ra * g.a.ld)) return cudaErrorInvalidValue;
  bool ok = encode(&p.a, false, a, operand_cols(g.a, g.m, g.k), ra, q.ld_a, f32 ? 3 : g.a.rest ? 2 : 1, ra, 64, p.a_k ? kTileM : kDeepK);
  ok = ok && encode(&p.b, false, b, operand_cols(g.b, g.n, g.k), rb, q.ld_b, f32 ? 3 : 1, rb, 64, p.b_k ? kRowsB : kDeepK);
  p.bias = g.bias;
  p.residual = g.residual;
  p.ldr = g.ldr;
  p.act = g.act;
  p.c_ptr = g.c;
  p.ldc = g.ldc;
  p.pre_ptr = g.pre;
  p.ldp = g.ldp;
  p.marks = marks;
  p.call = call;
  p.part = q.part;
  p.ticket = reinterpret_cast<unsigned*>(words.at) + 64;
  p.status = words.status;
  const int size = f32 ? 4 : 2;
  p.tma_c = tma_rows(g.c, g.ldc, size);
  p.tma_pre = g.pre && tma_rows(g.pre, g.ldp, size);
  if (p.tma_c) ok = ok && encode(&p.c, f32, g.c, g.n, g.m, g.ldc, 1, g.m, 128 / size, 32);
  if (p.tma_pre) ok = ok && encode(&p.pre, f32, g.pre, g.n, g.m, g.ldp, 1, g.m, 128 / size, 32);
  if (!ok) return cudaErrorInvalidValue;
  if (f32) return launch_mma_t<float, kTermsF32>(p, st);
  return g.a.rest ? launch_mma_t<__nv_bfloat16, kTermsRest>(p, st) : launch_mma_t<__nv_bfloat16, 1>(p, st);
}

}  // namespace tk

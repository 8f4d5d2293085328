// Matrix products c = act(a b^T + bias) + residual on the tensor cores
// (tcgen05.mma, bf16 operands, f32 accumulators in tensor memory).
//
// A persistent grid of CTAs (alone, or in pairs that share one product) takes
// work units (tile of c, part of k) in turn.  In each CTA one thread brings
// the operands' slices into a ring of shared-memory stages by TMA (128-byte
// swizzle, zeros outside the matrices), one thread of the (leading) CTA
// issues the products from them, and eight warps read finished accumulators
// from tensor memory, apply bias, activation and residual in f32, round once
// and store.  Tensor memory holds two accumulators, so that a tile's results
// are written while the next tile is multiplied.  When there are too few
// tiles for the GPU, k is cut into parts whose f32 sums go to scratch; a
// second kernel adds them in their order and applies the same epilogue.
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

template <int CTAS, int BN>
struct Shape {
  static constexpr int kRowsB = BN / CTAS;  // rows of b that one CTA brings in
  static constexpr int kBytesA = kTileM * kDeepK * 2, kBytesB = kRowsB * kDeepK * 2;
  static constexpr int kStage = kBytesA + kBytesB;
  static constexpr int kStages = 196608 / kStage;
  static constexpr int kOffStaging = kStages * kStage;
  static constexpr int kOffBias = kOffStaging + kEpiWarps * kStageBytesOut;
  static constexpr int kOffBars = kOffBias + 2 * BN * 4;
  static constexpr int kSmem = kOffBars + (2 * kStages + 4) * 8 + 16;
  static constexpr int kTmemCols = 2 * BN;
};

struct MmaParams {
  CUtensorMap a, b, c, pre;
  int64_t m, n;
  int k_blocks;            // stages along k
  int splits, k_per_split; // parts of k, stages of each
  int tiles_m, tiles_n;
  bool a_k, b_k;           // operand order: k contiguous
  uint32_t idesc;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  int64_t ldr;
  int act;
  bool tma_c, tma_pre;     // stores by TMA (else by plain stores)
  void* c_ptr;
  int64_t ldc;
  void* pre_ptr;
  int64_t ldp;
  bool want_pre;
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
template <int CTAS>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
               ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if constexpr (CTAS == 2) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  } else {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  }
}
template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, bool add) {
  if constexpr (CTAS == 2)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(uint32_t(add)) : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
// Arrives on `bar` (at the same place in each CTA) when the products issued so far are done.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"(uint16_t(3)) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
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

struct Unit {
  int m, n, split;  // tile and part of k
};
// Tiles in strips of kStrip tile rows, down the strip first: CTAs that run at
// the same time share rows of b and keep a strip of a in L2.
constexpr int kStrip = 16;
__device__ __forceinline__ Unit unit_of(int u, const MmaParams& p) {
  const int tiles = p.tiles_m * p.tiles_n;
  Unit r;
  r.split = u / tiles;
  const int t = u - r.split * tiles;
  const int strip = t / (kStrip * p.tiles_n);
  const int first = strip * kStrip;
  const int tall = min(kStrip, p.tiles_m - first);
  const int in = t - strip * kStrip * p.tiles_n;
  r.m = first + in % tall;
  r.n = in / tall;
  return r;
}

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
__device__ __forceinline__ void stage_residual(uint32_t staging, const __nv_bfloat16* src, int64_t ld, int64_t row0,
                                               int64_t rows, int64_t col0, int64_t cols, int lane) {
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = e * 32 + lane;
      uint16_t u = 0;
      if (row0 + r < rows && col0 + c < cols) u = __bfloat16_as_ushort(src[(row0 + r) * ld + col0 + c]);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(piece(staging, r, c / 8) + (c % 8) * 2), "h"(u) : "memory");
    }
  }
}
// 64 values of the lane's row, rounded to bf16, into staging.
__device__ __forceinline__ void stage_bf16(uint32_t staging, int lane, const float* v) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    Vec<__nv_bfloat16, 8> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = v[q * 8 + i];
    const uint4 u = o.pack();
    st_shared16(piece(staging, lane, q), u.x, u.y, u.z, u.w);
  }
}
template <int N>
__device__ __forceinline__ void apply_act(float* v, int act) {
  if (act == kActNone) return;
  if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value(v[i], kActRelu);
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value(v[i], kActGelu);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value(v[i], kActSilu);
  }
}

// PARTIAL: f32 sums of one part of k (no epilogue) to scratch; else bf16 results.
template <int CTAS, int BN, bool PARTIAL>
__global__ void __launch_bounds__(kThreads, 1) mma_kernel(const __grid_constant__ MmaParams p) {
  using S = Shape<CTAS, BN>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_addr(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  const uint32_t bars = base + S::kOffBars;
  auto full = [&](int s) { return bars + s * 8; };
  auto empty = [&](int s) { return bars + (S::kStages + s) * 8; };
  auto acc_full = [&](int b) { return bars + (2 * S::kStages + b) * 8; };
  auto acc_empty = [&](int b) { return bars + (2 * S::kStages + 2 + b) * 8; };
  const uint32_t tmem_word = bars + (2 * S::kStages + 4) * 8;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      bar_init(full(s), CTAS);  // each CTA's loads
      bar_init(empty(s), 1);    // the products that read the stage
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(acc_full(b), 1);
      bar_init(acc_empty(b), CTAS * kEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc<CTAS>(tmem_word, S::kTmemCols);
  fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();
  fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_word) : "memory");

  const int units = p.tiles_m * p.tiles_n * p.splits;
  const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {  // loads
      int stage = 0;
      uint32_t phase = 0;
      for (int u = first; u < units && ok; u += step) {
        const Unit w = unit_of(u, p);
        const int m0 = (w.m * CTAS + static_cast<int>(rank)) * kTileM;
        const int n0 = w.n * BN + static_cast<int>(rank) * S::kRowsB;
        const int kb0 = w.split * p.k_per_split, kb1 = min(p.k_blocks, kb0 + p.k_per_split);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = bar_wait(empty(stage), phase ^ 1))) break;
          const uint32_t sa = base + stage * S::kStage, sb = sa + S::kBytesA;
          const uint32_t bar = CTAS == 2 ? map_to_rank(full(stage), 0) : full(stage);
          bar_expect(bar, S::kStage);
          const int k0 = kb * kDeepK;
          if (p.a_k) {
            tma_load<CTAS>(sa, &p.a, k0, m0, bar);
          } else {
            tma_load<CTAS>(sa, &p.a, m0, k0, bar);
            tma_load<CTAS>(sa + 8192, &p.a, m0 + 64, k0, bar);
          }
          if (p.b_k) {
            tma_load<CTAS>(sb, &p.b, k0, n0, bar);
          } else {
#pragma unroll
            for (int i = 0; i < S::kRowsB / 64; ++i) tma_load<CTAS>(sb + i * 8192, &p.b, n0 + i * 64, k0, bar);
          }
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // every stage has been read before this CTA ends
      for (int s = 0; s < S::kStages && ok; ++s) {
        ok = bar_wait(empty(stage), phase ^ 1);
        if (++stage == S::kStages) {
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
      for (int u = first; u < units && ok; u += step) {
        const Unit w = unit_of(u, p);
        const int kb0 = w.split * p.k_per_split, kb1 = min(p.k_blocks, kb0 + p.k_per_split);
        if (!(ok = bar_wait(acc_empty(buf), acc_phase ^ 1))) break;
        fence_after();
        const uint32_t d = tmem + buf * BN;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = bar_wait(full(stage), phase))) break;
          fence_after();
          const uint32_t sa = base + stage * S::kStage, sb = sa + S::kBytesA;
          const uint64_t da = operand_desc(sa, 8192), db = operand_desc(sb, 8192);
#pragma unroll
          for (int i = 0; i < kDeepK / 16; ++i)
            mma<CTAS>(d, da + i * step_a, db + i * step_b, p.idesc, kb > kb0 || i > 0);
          mma_commit<CTAS>(empty(stage));
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        mma_commit<CTAS>(acc_full(buf));
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1;
      }
    }
  } else if (warp >= 4) {  // results
    const int e = warp - 4, quad = e % 4, half = e / 4;
    const uint32_t staging = base + S::kOffStaging + e * kStageBytesOut;
    float* bias_smem = reinterpret_cast<float*>(smem + S::kOffBias);
    constexpr int kChunk = PARTIAL ? 32 : 64;  // columns of 128 bytes
    constexpr int kHalf = BN / 2;
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < units; u += step) {
      const Unit w = unit_of(u, p);
      const int64_t row0 = int64_t(w.m * CTAS + static_cast<int>(rank)) * kTileM + quad * 32;
      const int64_t n0 = int64_t(w.n) * BN;
      if constexpr (!PARTIAL) {
        if (p.bias) {
          for (int i = threadIdx.x - 128; i < BN; i += 32 * kEpiWarps)
            bias_smem[buf * BN + i] = n0 + i < p.n ? to_f32(p.bias[n0 + i]) : 0.0f;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
      }
      // (a warp that gave up goes on without waiting, so that the others' barriers are still met)
      if (ok) ok = __all_sync(~0u, bar_wait(acc_full(buf), acc_phase));
      fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < kHalf; c0 += kChunk) {
        float v[kChunk];
        const uint32_t from = tmem + buf * BN + half * kHalf + c0 + (uint32_t(quad * 32) << 16);
#pragma unroll
        for (int i = 0; i < kChunk; i += 32) tmem_load32(from + i, v + i);
        tmem_wait_load();
        if (c0 + kChunk == kHalf) {  // the accumulator is free
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(CTAS == 2 ? map_to_rank(acc_empty(buf), 0) : acc_empty(buf));
        }
        const int64_t col0 = n0 + half * kHalf + c0;
        if (lane == 0) store_wait_read();  // the staging's last store has been read
        __syncwarp();
        if constexpr (PARTIAL) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared16(piece(staging, lane, q), __float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                        __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && col0 < p.n && row0 < p.m) {
            tma_store(&p.c, static_cast<int>(col0), static_cast<int>(row0), w.split, staging);
            store_commit();
          }
        } else {
          if (p.bias) {
            const float4* b = reinterpret_cast<const float4*>(bias_smem + buf * BN + half * kHalf + c0);
#pragma unroll
            for (int i = 0; i < kChunk / 4; ++i) {
              const float4 t = b[i];
              v[4 * i] += t.x;
              v[4 * i + 1] += t.y;
              v[4 * i + 2] += t.z;
              v[4 * i + 3] += t.w;
            }
          }
          if (p.want_pre) {
            stage_bf16(staging, lane, v);
            fence_proxy_async_smem();
            __syncwarp();
            if (p.tma_pre) {
              if (lane == 0 && col0 < p.n && row0 < p.m) {
                tma_store(&p.pre, static_cast<int>(col0), static_cast<int>(row0), 0, staging);
                store_commit();
                store_wait_read();
              }
            } else {
              store_plain(staging, static_cast<__nv_bfloat16*>(p.pre_ptr), p.ldp, row0, p.m, col0, p.n, lane);
            }
            __syncwarp();
          }
          apply_act<kChunk>(v, p.act);
          if (p.residual) {
            stage_residual(staging, p.residual, p.ldr, row0, p.m, col0, p.n, lane);
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              Vec<__nv_bfloat16, 8> r;
              r.set(ld_shared16(piece(staging, lane, q)));
#pragma unroll
              for (int i = 0; i < 8; ++i) v[q * 8 + i] += r.v[i];
            }
          }
          stage_bf16(staging, lane, v);
          fence_proxy_async_smem();
          __syncwarp();
          if (p.tma_c) {
            if (lane == 0 && col0 < p.n && row0 < p.m) {
              tma_store(&p.c, static_cast<int>(col0), static_cast<int>(row0), 0, staging);
              store_commit();
            }
          } else {
            store_plain(staging, static_cast<__nv_bfloat16*>(p.c_ptr), p.ldc, row0, p.m, col0, p.n, lane);
          }
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
  if constexpr (CTAS == 2) cluster_sync();
  fence_after();
  if (warp == 2) tmem_free<CTAS>(tmem, S::kTmemCols);
}

// Adds the parts of k in their order, and the epilogue.
__global__ void __launch_bounds__(256) join_parts_kernel(const float* part, int64_t stride, int64_t ld, int splits, int64_t m,
                                                         int64_t n, const __nv_bfloat16* bias,
                                                         const __nv_bfloat16* residual, int64_t ldr, int act,
                                                         __nv_bfloat16* c, int64_t ldc, __nv_bfloat16* pre, int64_t ldp) {
  const int64_t quads = (n + 3) / 4;
  const int64_t at = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (at >= m * quads) return;
  const int64_t i = at / quads, j = (at - i * quads) * 4;
  float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float* src = part + i * ld + j;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(src + s * stride));
    z.x += t.x;
    z.y += t.y;
    z.z += t.z;
    z.w += t.w;
  }
  const float zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (j + e >= n) break;
    float v = zs[e] + (bias ? to_f32(bias[j + e]) : 0.0f);
    if (pre) pre[i * ldp + j + e] = from_f32<__nv_bfloat16>(v);
    v = act_value(v, act);
    if (residual) v += to_f32(residual[i * ldr + j + e]);
    c[i * ldc + j + e] = from_f32<__nv_bfloat16>(v);
  }
}

// Copies an operand whose rows TMA cannot address to rows of `ld` values (a multiple of 8).
__global__ void __launch_bounds__(256) align_rows_kernel(const __nv_bfloat16* src, int64_t lds, int64_t rows, int64_t cols,
                                                         __nv_bfloat16* dst, int64_t ld) {
  const int64_t per = (cols + 255) / 256;
  const int64_t r = blockIdx.x / per, c = (blockIdx.x % per) * 256 + threadIdx.x;
  if (r < rows && c < cols) dst[r * ld + c] = src[r * lds + c];
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
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes ? 3 : 2, const_cast<void*>(p),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tma_rows(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

struct MmaPlan {
  int shape;  // 0: pair, 256 x 256; 1: pair, 256 x 128; 2: one CTA, 128 x 128
  int tiles_m, tiles_n, k_blocks, splits, k_per_split;
  int64_t part_ld, part_rows;
  __nv_bfloat16* copy_a;
  __nv_bfloat16* copy_b;
  int64_t ld_a, ld_b;
  float* part;
};
constexpr int kShapeCtas[3] = {2, 2, 1}, kShapeN[3] = {256, 128, 128};

int64_t operand_rows(const Operand& o, int64_t i, int64_t k) { return o.k_inner ? i : k; }
int64_t operand_cols(const Operand& o, int64_t i, int64_t k) { return o.k_inner ? k : i; }

MmaPlan plan_mma(const Product& g, Scratch& sc) {
  MmaPlan q{};
  q.k_blocks = static_cast<int>((g.k + kDeepK - 1) / kDeepK);
  q.shape = 0;
  q.splits = 1;
  const int sms = ops_sm_count();
  double best = 1e30;
  for (int shape = 0; shape < 3; ++shape) {
    const int64_t tm = (g.m + kTileM * kShapeCtas[shape] - 1) / (kTileM * kShapeCtas[shape]);
    const int64_t tn = (g.n + kShapeN[shape] - 1) / kShapeN[shape];
    const int64_t slots = sms / kShapeCtas[shape];
    const double per_block = shape == 0 ? 512 : shape == 1 ? 320 : 400;  // cycles a stage
    if (tm * tn > INT32_MAX / 64) continue;
    for (int s = 1; s <= 16 && s <= q.k_blocks; ++s) {
      const int64_t kp = (q.k_blocks + s - 1) / s;
      if ((q.k_blocks + kp - 1) / kp != s) continue;
      const double waves = static_cast<double>((tm * tn * s + slots - 1) / slots);
      const double join = s == 1 ? 0 : 5000.0 + 8.0 * s * g.m * g.n / 2500.0;
      const double t = waves * (kp * per_block + 700.0) + join;
      if (t < best) {
        best = t;
        q.shape = shape;
        q.splits = s;
        q.k_per_split = static_cast<int>(kp);
        q.tiles_m = static_cast<int>(tm);
        q.tiles_n = static_cast<int>(tn);
      }
    }
  }
  const bool ta = tma_rows(g.a.p, g.a.ld), tb = tma_rows(g.b.p, g.b.ld);
  q.ld_a = g.a.ld;
  q.ld_b = g.b.ld;
  if (!ta) {
    q.ld_a = (operand_cols(g.a, g.m, g.k) + 7) / 8 * 8;
    q.copy_a = sc.take<__nv_bfloat16>(q.ld_a * operand_rows(g.a, g.m, g.k));
  }
  if (!tb) {
    q.ld_b = (operand_cols(g.b, g.n, g.k) + 7) / 8 * 8;
    q.copy_b = sc.take<__nv_bfloat16>(q.ld_b * operand_rows(g.b, g.n, g.k));
  }
  if (q.splits > 1) {
    q.part_ld = (g.n + 3) / 4 * 4;
    q.part_rows = g.m;
    q.part = sc.take<float>(q.part_ld * q.part_rows * q.splits);
  }
  return q;
}

template <int CTAS, int BN, bool PARTIAL>
cudaError_t launch_shape(const MmaParams& p, cudaStream_t st) {
  using S = Shape<CTAS, BN>;
  static_assert(S::kSmem <= 232448, "shared memory of one CTA");
  auto kernel = mma_kernel<CTAS, BN, PARTIAL>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int units = p.tiles_m * p.tiles_n * p.splits;
  const int slots = ops_sm_count() / CTAS;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((units < slots ? units : slots) * CTAS));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool PARTIAL>
cudaError_t launch_any(int shape, const MmaParams& p, cudaStream_t st) {
  switch (shape) {
    case 0: return launch_shape<2, 256, PARTIAL>(p, st);
    case 1: return launch_shape<2, 128, PARTIAL>(p, st);
    default: return launch_shape<1, 128, PARTIAL>(p, st);
  }
}

cudaError_t align_rows(const Operand& o, int64_t i, int64_t k, __nv_bfloat16* dst, int64_t ld, cudaStream_t st) {
  const int64_t rows = operand_rows(o, i, k), cols = operand_cols(o, i, k);
  const int64_t blocks = rows * ((cols + 255) / 256);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  align_rows_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(o.p), o.ld, rows, cols, dst, ld);
  return cudaGetLastError();
}

}  // namespace

size_t mma_scratch_bytes(const Product& g) {
  Scratch sc;
  plan_mma(g, sc);
  return sc.used();
}

cudaError_t launch_mma(const Product& g, Scratch& sc, int* status, cudaStream_t st) {
  const MmaPlan q = plan_mma(g, sc);
  if (!q.tiles_m) return cudaErrorInvalidValue;  // more tiles than a launch counts
  cudaError_t e = cudaSuccess;
  if (q.copy_a) e = align_rows(g.a, g.m, g.k, q.copy_a, q.ld_a, st);
  if (e == cudaSuccess && q.copy_b) e = align_rows(g.b, g.n, g.k, q.copy_b, q.ld_b, st);
  if (e != cudaSuccess) return e;
  MmaParams p{};
  p.m = g.m;
  p.n = g.n;
  p.k_blocks = q.k_blocks;
  p.splits = q.splits;
  p.k_per_split = q.k_per_split;
  p.tiles_m = q.tiles_m;
  p.tiles_n = q.tiles_n;
  p.a_k = g.a.k_inner;
  p.b_k = g.b.k_inner;
  const int ctas = kShapeCtas[q.shape], bn = kShapeN[q.shape];
  // f32 accumulators, bf16 operands, their order, and the product's size
  p.idesc = (1u << 4) | (1u << 7) | (1u << 10) | (p.a_k ? 0u : 1u << 15) | (p.b_k ? 0u : 1u << 16) |
            (static_cast<uint32_t>(bn / 8) << 17) | (static_cast<uint32_t>(kTileM * ctas / 16) << 24);
  const void* a = q.copy_a ? q.copy_a : g.a.p;
  const void* b = q.copy_b ? q.copy_b : g.b.p;
  bool ok = p.a_k ? encode(&p.a, false, a, g.k, g.m, q.ld_a, 0, 0, kDeepK, kTileM)
                  : encode(&p.a, false, a, g.m, g.k, q.ld_a, 0, 0, 64, kDeepK);
  ok = ok && (p.b_k ? encode(&p.b, false, b, g.k, g.n, q.ld_b, 0, 0, kDeepK, bn / ctas)
                    : encode(&p.b, false, b, g.n, g.k, q.ld_b, 0, 0, 64, kDeepK));
  p.status = status;
  if (q.splits > 1) {
    ok = ok && encode(&p.c, true, q.part, q.part_ld, q.part_rows, q.part_ld, q.splits, q.part_rows, 32, 32);
    if (!ok) return cudaErrorInvalidValue;
    p.tma_c = true;
    e = launch_any<true>(q.shape, p, st);
    if (e != cudaSuccess) return e;
    const int64_t quads = (g.n + 3) / 4;
    const int64_t blocks = (g.m * quads + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    join_parts_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
        q.part, q.part_ld * q.part_rows, q.part_ld, q.splits, g.m, g.n, static_cast<const __nv_bfloat16*>(g.bias),
        static_cast<const __nv_bfloat16*>(g.residual), g.ldr, g.act, static_cast<__nv_bfloat16*>(g.c), g.ldc,
        static_cast<__nv_bfloat16*>(g.pre), g.ldp);
    return cudaGetLastError();
  }
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.residual = static_cast<const __nv_bfloat16*>(g.residual);
  p.ldr = g.ldr;
  p.act = g.act;
  p.c_ptr = g.c;
  p.ldc = g.ldc;
  p.pre_ptr = g.pre;
  p.ldp = g.ldp;
  p.want_pre = g.pre != nullptr;
  p.tma_c = tma_rows(g.c, g.ldc);
  p.tma_pre = g.pre && tma_rows(g.pre, g.ldp);
  if (p.tma_c) ok = ok && encode(&p.c, false, g.c, g.n, g.m, g.ldc, 1, g.m, 64, 32);
  if (p.tma_pre) ok = ok && encode(&p.pre, false, g.pre, g.n, g.m, g.ldp, 1, g.m, 64, 32);
  if (!ok) return cudaErrorInvalidValue;
  return launch_any<false>(q.shape, p, st);
}

}  // namespace tk

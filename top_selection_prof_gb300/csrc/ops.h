// Internal interface of the operators around the selection (the linear layer,
// the products of a selection with a dictionary, the gradient norm; a language
// model's tokens, experts and cache): host declarations shared by their C entries (ops_api.cu) and their kernels.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace tk {

// Scratch of one call, carved from the operators' per-(device, stream) block:
// 256-byte aligned pieces handed out in order.  `plan` only adds up sizes, so
// a call lays itself out once to know its size and once to take its pointers.
class Scratch {
 public:
  explicit Scratch(void* base = nullptr) : base_(static_cast<char*>(base)) {}
  template <typename T>
  T* take(int64_t count) {
    const size_t at = used_;
    used_ += (sizeof(T) * static_cast<size_t>(count < 1 ? 1 : count) + 255) & ~size_t(255);
    return base_ ? reinterpret_cast<T*>(base_ + at) : nullptr;
  }
  size_t used() const { return used_; }

 private:
  char* base_;
  size_t used_ = 0;
};

// Status of the operators' device waits on `st` since it was last asked (the
// stream must have been synchronised): kDevOk or kDevTimeout.
cudaError_t ops_take_status(cudaStream_t st, int* status);

// Words that each (device, stream) keeps for the operators, zero at first, as
// those of a captured call are at each replay: [0] the status that a kernel sets
// when a wait runs out, [32] and [64..] tickets that every kernel leaves at zero,
// [kOpsMarks..] what the operands of the tensor cores' products hold.
constexpr int64_t kOpsWords = 16384, kOpsMarks = 48;
// Each mark is the number of the last call that found: a value that is not finite (or not as bf16), a value of a or of b
// too small for parts (f32 only), a value of either too large to be scaled.
enum : int { kMarkOther = 0, kMarkSmallA = 1, kMarkSmallB = 2, kMarkLarge = 3 };

struct Words {
  int* at = nullptr;      // kOpsWords
  int* status = nullptr;  // where a wait that runs out is told
};

// A number found once for each device (0: not yet).
class PerDevice {
 public:
  // The current device's number; null when there is no telling it apart.
  std::atomic<int>* here() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMost ? &of_[dev] : nullptr;
  }

 private:
  static constexpr int kMost = 64;
  std::atomic<int> of_[kMost] = {};
};

// SMs of the current device.
int ops_sm_count();

// ---- linear (kernels_linear.cu) ----------------------------------------------
enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

// A matrix operand of a product over a shared index k: element (i, k) at
// p[i * ld + k] when k_inner, else at p[k * ld + i].  An operand a of bf16
// values may hold more bits than they have: what their rounding left, rounded
// in its turn, then lies `rest` values further on (rows on 16-byte boundaries).
struct Operand {
  const void* p;
  int64_t ld;
  bool k_inner;
  int64_t rest = 0;  // 0: none
};
// c[i, j] = act(sum_k a(i, k) b(j, k) + bias[j]) + residual[i, j]; the value
// before act is written to pre when that is not null.  All of one dtype.
struct Product {
  Operand a, b;
  int64_t m, n, k;
  int dtype;
  const void* bias;      // nullable, n values
  const void* residual;  // nullable
  int64_t ldr;
  int act;
  void* c;
  int64_t ldc;
  void* pre;             // nullable
  int64_t ldp;
};
cudaError_t launch_product(const Product& g, Scratch& sc, const Words& words, cudaStream_t st);
size_t product_scratch_bytes(const Product& g);
// The same on the tensor cores (kernels_mma.cu), or by launch_simt's kernel where the marks that `call` leaves say so.
cudaError_t launch_mma(const Product& g, Scratch& sc, const Words& words, int call, cudaStream_t st);
cudaError_t launch_simt(const Product& g, const int* marks, int call, cudaStream_t st);
size_t mma_scratch_bytes(const Product& g);

// dz = dy * act'(pre) (act != none) and the column sums of dz into dbias
// (nullable).  With act == none only the sums are formed, from dy.  bf16: what
// dz's rounding left goes, rounded, to dz + rest (0: not wanted).
struct SlopeSums {
  const void* dy;
  int64_t lddy;
  const void* pre;
  int64_t ldp;
  int dtype;
  int64_t rows, n;
  int act;
  void* dz;     // nullable with act == none
  int64_t lddz, rest;
  void* dbias;  // nullable
  float* part;  // slope_sums_parts(rows, n) * n values, when dbias is wanted
};
int64_t slope_sums_parts(int64_t rows, int64_t n);
cudaError_t launch_slope_sums(const SlopeSums& s, cudaStream_t st);

// ---- products of a selection (kernels_places.cu) ------------------------------
// The selected places, as the selection returns them: flat positions r*n + c
// (per_row == 0, `count` of them), or `count` row-local positions c for each
// row.  Positions out of range (-1 where a selection returned fewer) hold no place.
struct Places {
  const int64_t* idx;
  int64_t count;
  bool per_row;
  int64_t rows, n;
  int64_t total;  // places in all
};
// Coefficient of place s: coef[s] (0 where coef is null), or 0 where gate is given and gate[s] <= 0 or NaN.
struct Coef {
  const void* coef;
  const void* gate;  // nullable
};
// y[r] = bias + sum over the places of row r of coef_s * w[c_s]   (d values a row)
struct RowSums {
  Places places;
  Coef coef;
  int dtype;
  const void* w;
  int64_t ldw, d;
  const void* bias;  // nullable
  void* y;           // contiguous
};
// For each column c: dw[c] = sum over its places of coef_s * x[r_s]; dbias[c] =
// sum of coef_s; and for each of its places dots[s] = <x[r_s], w[c]>.
struct ColumnSums {
  Places places;
  Coef coef;
  int dtype;
  const void* x;
  int64_t ldx, d;
  const void* w;  // with dots
  int64_t ldw;
  void* dw;       // nullable, contiguous
  void* dbias;    // nullable, n values
  void* dots;     // nullable, one a place (0 where a position is out of range)
};
// Either or both (null: not wanted; both over the same places and coefficients).
size_t sums_scratch_bytes(const ColumnSums* c, const RowSums* r);
cudaError_t launch_sums(const ColumnSums* c, const RowSums* r, Scratch& sc, cudaStream_t st);

// ---- gradient norm (kernels_norm.cu) --------------------------------------------
struct ClipTensor {
  const void* in;
  void* out;  // null: norm only
  int64_t count;
  int dtype;
};
size_t clip_scratch_bytes();
// scale == false: the norm alone.
cudaError_t launch_clip(const ClipTensor* t, int64_t num, bool scale, float max_norm, float* norm, const Words& words,
                        Scratch& sc, cudaStream_t st);

// ---- tokens from logits (kernels_tokens.cu) ------------------------------------
constexpr int64_t kTokensMaxLen = int64_t(1) << 18;
// Each parameter is one number, or one a row where its pointer is not null.
struct TokenDraw {
  const void* x;
  int64_t ld;
  int dtype;
  int64_t rows;
  int n;
  const float* u;
  float temperature, top_p, min_p;
  int top_k;
  const float *temperatures, *top_ps, *min_ps;
  const int32_t* top_ks;
  int64_t* tokens;
  float* logprobs;
  double per, log_min_p;  // log2(e) / temperature and ln(min_p) of the numbers
};
cudaError_t launch_tokens(const TokenDraw& p, cudaStream_t st);

// ---- rows by expert and back (kernels_experts.cu) ------------------------------
constexpr int64_t kMostExperts = 4096;
struct Dispatch {
  const void* x;
  int64_t ldx;
  const int64_t* idx;
  int64_t tokens, k, experts, d;
  int dtype;
  void* xs;
  int64_t* place;
  int64_t* offsets;
};
size_t dispatch_scratch_bytes(const Dispatch& p);
cudaError_t launch_dispatch(const Dispatch& p, Scratch& sc, cudaStream_t st);
// y, or from dy: dys and dweights (each nullable).
struct Combine {
  const void* ys;
  int64_t ldys, rows;
  const int64_t* place;
  const void* weights;  // nullable
  int64_t tokens, k, d;
  int dtype;
  void* y;
  const void* dy;
  int64_t lddy;
  void* dys;
  void* dweights;
};
cudaError_t launch_combine(const Combine& p, cudaStream_t st);
size_t combine_backward_scratch_bytes(const Combine& p);
cudaError_t launch_combine_backward(const Combine& p, Scratch& sc, cudaStream_t st);

// ---- what stays in a cache (kernels_cache.cu) ----------------------------------
// Rows of contiguous values: distances, in elements, between batches, heads and rows.
struct View {
  void* data;
  int64_t batch, head, row;
};
struct Evict {
  View keys, values;  // batch, head, position
  View score;         // f32; batch, head (positions are contiguous)
  const int64_t* lengths;
  View weights;       // batch, query head, query (positions are contiguous); data may be null
  int weights_dtype;
  int64_t group, queries;
  int dtype;
  int64_t batch, heads, capacity, key_dim, value_dim, keep, recent;
  void *out_keys, *out_values;
  float* out_score;
  int64_t *out_kept, *out_lengths;
};
size_t evict_scratch_bytes(const Evict& p);
cudaError_t launch_evict(const Evict& p, Scratch& sc, cudaStream_t st);
struct Replace {
  View keys, values, score, positions;  // in place
  const int64_t* lengths;
  View key, value;    // batch, head
  View weights;
  int weights_dtype;
  int64_t group, queries;
  int dtype;
  int64_t batch, heads, capacity, key_dim, value_dim, recent;
  int64_t* slots;
};
cudaError_t launch_replace(const Replace& p, cudaStream_t st);

}  // namespace tk

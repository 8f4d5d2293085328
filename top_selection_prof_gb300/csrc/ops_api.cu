// C entries of the operators around the selection (declared in include/topk.h):
// argument checks, the per-(device, stream) scratch block and the launches.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <map>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "../../include/topk.h"
#include "common.cuh"
#include "engine.h"
#include "ops.h"

namespace tk {

int ops_sm_count() {
  static PerDevice sms;
  std::atomic<int>* n = sms.here();
  int dev = 0, v = n ? n->load() : 0;
  if (v) return v;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
  if (n) *n = v;
  return v;
}

namespace {

// cudaErrorNotSupported: more blocks or tiles than a launch counts.
int status_of(cudaError_t e) {
  if (e == cudaSuccess) return TOPK_OK;
  cudaGetLastError();  // (reported here, not to the caller's next CUDA call)
  return e == cudaErrorMemoryAllocation ? TOPK_ENOMEM : e == cudaErrorNotSupported ? TOPK_EUNSUPPORTED : TOPK_ECUDA;
}

// Scratch blocks of the operators, apart from the selection's (which keeps
// words at zero between calls).  Grown with stream-ordered allocation, the old
// block released in stream order, never shrunk.
struct Block {
  void* ptr = nullptr;
  size_t bytes = 0;
  int* words = nullptr;  // kOpsWords
};
std::mutex g_mu;
std::map<StreamKey, Block> g_blocks;

// One call's use of its stream's block: the stream is held until the call's
// last launch is enqueued.  A call that is captured into a graph has a block of
// its own, made and released by the graph: the stream's block may be replaced
// while the graph lives, and the graph may be replayed beside the stream's calls.
class Call {
 public:
  explicit Call(cudaStream_t st) : st_(st), key_error_(stream_key(st, &key_)), hold_(key_) {}
  cudaError_t scratch(size_t bytes, void** out, Words* words = nullptr) {
    if (key_error_ != cudaSuccess) return key_error_;
    cudaStreamCaptureStatus capture;
    const cudaError_t asked = cudaStreamIsCapturing(st_, &capture);
    if (asked != cudaSuccess) return asked;
    std::unique_lock<std::mutex> lock(g_mu);
    Block& b = g_blocks[key_];  // (nodes do not move; this one is the holder's)
    lock.unlock();
    cudaError_t e = cudaSuccess;
    if (capture != cudaStreamCaptureStatusNone) {
      const size_t head = words ? sizeof(int) * kOpsWords : 0;
      *out = nullptr;
      if (!head && !bytes) return cudaSuccess;
      e = cudaMallocAsync(&graph_, head + bytes, st_);
      if (e != cudaSuccess) {
        graph_ = nullptr;
        return e;
      }
      *out = static_cast<char*>(graph_) + head;
      if (!words) return cudaSuccess;
      words->at = static_cast<int*>(graph_);
      words->status = b.words ? b.words : words->at;  // (a word that topk_last_status finds, if there is one)
      return cudaMemsetAsync(graph_, 0, head, st_);
    }
    if (b.bytes < bytes) {
      const size_t grow = (bytes + bytes / 4 + 0xFFFFF) & ~size_t(0xFFFFF);
      void* p = nullptr;
      e = cudaMallocAsync(&p, grow, st_);
      if (e != cudaSuccess) return e;
      if (b.ptr) e = cudaFreeAsync(b.ptr, st_);
      b.ptr = p;
      b.bytes = grow;
      if (e != cudaSuccess) return e;
    }
    if (words && !b.words) {
      int* w = nullptr;
      e = cudaMallocAsync(&w, sizeof(int) * kOpsWords, st_);
      if (e == cudaSuccess) e = cudaMemsetAsync(w, 0, sizeof(int) * kOpsWords, st_);
      if (e != cudaSuccess) return e;
      b.words = w;
    }
    *out = b.ptr;
    if (words) *words = Words{b.words, b.words};
    return cudaSuccess;
  }
  // The status of a call whose launches gave e.
  int end(cudaError_t e) {
    if (graph_) {
      const cudaError_t released = cudaFreeAsync(graph_, st_);
      if (e == cudaSuccess) e = released;
    }
    return status_of(e);
  }

 private:
  cudaStream_t st_;
  StreamKey key_;
  cudaError_t key_error_;
  StreamHold hold_;
  void* graph_ = nullptr;
};

// No exception leaves a C entry: the library's own containers can only run out of host memory.
template <typename F>
int guarded(F f) noexcept {
  try {
    return f();
  } catch (...) {
    return TOPK_ENOMEM;
  }
}

bool known_dtype(int dtype) { return dtype == TOPK_F32 || dtype == TOPK_BF16; }
bool known_act(int act) { return act >= TOPK_ACT_NONE && act <= TOPK_ACT_SILU; }
constexpr int64_t kMaxExtent = INT32_MAX;
size_t value_bytes(int dtype) { return dtype == TOPK_F32 ? 4 : 2; }

// Where a matrix lies: `rows` runs of `row` bytes, `ld` bytes from one to the next (0: there is one).  At null: none.
struct Span {
  uintptr_t at;
  int64_t rows, row, ld;
};
Span matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return {reinterpret_cast<uintptr_t>(p), rows, cols * size, rows > 1 ? ld * size : 0};
}
Span vector(const void* p, int64_t n, int64_t size) { return matrix(p, 1, n, n, size); }
// Whether two matrices have a byte in common; those whose rows lie differently far apart count as having one wherever their
// ranges meet.
bool meet(Span a, Span b) {
  if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.row < 1 || b.row < 1) return false;
  if (b.at < a.at) std::swap(a, b);
  if (b.at - a.at >= static_cast<uintptr_t>((a.rows - 1) * a.ld + a.row)) return false;
  if (a.rows == 1 || (b.rows > 1 && a.ld != b.ld)) return true;
  // b begins in a run of a, or in the gap before the next one
  const int64_t d = static_cast<int64_t>((b.at - a.at) % static_cast<uintptr_t>(a.ld));
  return d < a.row || d + b.row > a.ld;
}
// Whether an output has a byte in common with an input or another output.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return true;
    for (auto p = outs.begin(); p != o; ++p)
      if (meet(*o, *p)) return true;
  }
  return false;
}

int linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, const void* residual, int64_t ldr,
           int dtype, int64_t rows, int64_t inner, int64_t outer, int act, void* y, int64_t ldy, void* pre, int64_t ldp,
           cudaStream_t st) {
  if (!known_dtype(dtype) || !known_act(act) || rows < 0 || inner < 1 || outer < 1) return TOPK_EINVAL;
  if (rows == 0) return TOPK_OK;
  if (!x || !w || !y || ldx < inner || ldw < inner || ldy < outer) return TOPK_EINVAL;
  if ((residual && ldr < outer) || (pre && ldp < outer)) return TOPK_EINVAL;
  if (rows > kMaxExtent || inner > kMaxExtent || outer > kMaxExtent) return TOPK_EUNSUPPORTED;
  const int64_t size = static_cast<int64_t>(value_bytes(dtype));
  const Span my = matrix(y, rows, outer, ldy, size), mr = matrix(residual, rows, outer, ldr, size);
  // (in place: each value of the residual is read where its result is then written)
  const bool in_place = my.at == mr.at && (my.ld == mr.ld || rows == 1);
  if (clash({my, matrix(pre, rows, outer, ldp, size)},
            {matrix(x, rows, inner, ldx, size), matrix(w, outer, inner, ldw, size), vector(bias, outer, size)}) ||
      (!in_place && meet(my, mr)) || meet(matrix(pre, rows, outer, ldp, size), mr))
    return TOPK_EINVAL;
  const Product g{{x, ldx, true}, {w, ldw, true}, rows, outer, inner, dtype, bias, residual, ldr, act, y, ldy, pre, ldp};
  void* base = nullptr;
  Words words;
  Call call(st);
  cudaError_t e = call.scratch(product_scratch_bytes(g), &base, &words);
  if (e != cudaSuccess) return call.end(e);
  Scratch sc(base);
  return call.end(launch_product(g, sc, words, st));
}

int linear_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* pre,
                    int64_t ldp, int dtype, int64_t rows, int64_t inner, int64_t outer, int act, void* dx, void* dw,
                    void* dbias, cudaStream_t st) {
  if (!known_dtype(dtype) || !known_act(act) || rows < 0 || inner < 1 || outer < 1) return TOPK_EINVAL;
  if (!dx && !dw && !dbias) return TOPK_OK;
  if (rows > kMaxExtent || inner > kMaxExtent || outer > kMaxExtent) return TOPK_EUNSUPPORTED;
  if (rows == 0) {  // sums over no rows
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemsetAsync(dw, 0, value_bytes(dtype) * static_cast<size_t>(inner * outer), st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, value_bytes(dtype) * static_cast<size_t>(outer), st);
    return status_of(e);
  }
  if (!dy || lddy < outer || (dw && (!x || ldx < inner)) || (dx && (!w || ldw < inner))) return TOPK_EINVAL;
  if (act != TOPK_ACT_NONE && (!pre || ldp < outer)) return TOPK_EINVAL;
  const int64_t size = static_cast<int64_t>(value_bytes(dtype));
  if (clash({vector(dx, rows * inner, size), vector(dw, outer * inner, size), vector(dbias, outer, size)},
            {matrix(dy, rows, outer, lddy, size), matrix(act != TOPK_ACT_NONE ? pre : nullptr, rows, outer, ldp, size),
             matrix(dw ? x : nullptr, rows, inner, ldx, size), matrix(dx ? w : nullptr, outer, inner, ldw, size)}))
    return TOPK_EINVAL;
  SlopeSums s{dy, lddy, pre, ldp, dtype, rows, outer, act, nullptr, 0, 0, dbias, nullptr};
  const bool make_dz = act != TOPK_ACT_NONE && (dx || dw);
  // bf16: a smooth activation's dz has more bits than bf16 holds; a second array keeps eight more (half the error of the
  // gradients of 2000 x 4096 x 16384 would be dz's own rounding: 0.0023 of them against 0.0017)
  const int64_t lddz = (outer + 7) / 8 * 8;
  const bool parts = dtype == TOPK_BF16 && (act == TOPK_ACT_GELU || act == TOPK_ACT_SILU);
  Product gx{{dy, lddy, true}, {w, ldw, false}, rows, inner, outer, dtype, nullptr, nullptr, 0, kActNone, dx, inner, nullptr, 0};
  Product gw{{dy, lddy, false}, {x, ldx, false}, outer, inner, rows, dtype, nullptr, nullptr, 0, kActNone, dw, inner, nullptr, 0};
  auto lay = [&](Scratch& sc) {
    if (make_dz) {
      s.dz = sc.take<char>(static_cast<int64_t>(value_bytes(dtype)) * rows * lddz * (parts ? 2 : 1));
      s.lddz = lddz;
      s.rest = parts ? rows * lddz : 0;
      gx.a = Operand{s.dz, lddz, true, s.rest};
      gw.a = Operand{s.dz, lddz, false, s.rest};
    }
    if (dbias) s.part = sc.take<float>(slope_sums_parts(rows, outer) * outer);
  };
  Scratch plan;
  lay(plan);
  const size_t px = dx ? product_scratch_bytes(gx) : 0, pw = dw ? product_scratch_bytes(gw) : 0;
  void* base = nullptr;
  Words words;
  Call call(st);
  cudaError_t e = call.scratch(plan.used() + (px > pw ? px : pw), &base, &words);
  if (e != cudaSuccess) return call.end(e);
  Scratch sc(base);
  lay(sc);
  if (make_dz || dbias) e = launch_slope_sums(s, st);
  if (e == cudaSuccess && dx) {
    Scratch own = sc;
    e = launch_product(gx, own, words, st);
  }
  if (e == cudaSuccess && dw) {
    Scratch own = sc;
    e = launch_product(gw, own, words, st);
  }
  return call.end(e);
}

// Checks the places of a selection; TOPK_OK or the error.
int check_places(const int64_t* idx, int64_t count, int per_row, int dtype, int64_t rows, int64_t n, int64_t d) {
  if (!known_dtype(dtype) || rows < 0 || n < 1 || d < 1 || count < 0) return TOPK_EINVAL;
  if (rows > kMaxExtent || n > kMaxExtent || d > kMaxExtent) return TOPK_EUNSUPPORTED;
  if (per_row && count > 0 && rows > kMaxExtent / count) return TOPK_EUNSUPPORTED;
  if (count > kMaxExtent) return TOPK_EUNSUPPORTED;
  const int64_t total = per_row ? rows * count : count;
  if (total >= (int64_t(1) << 29)) return TOPK_EUNSUPPORTED;
  if (total > 0 && !idx) return TOPK_EINVAL;
  return TOPK_OK;
}

// Runs the sums by column and by row and the column sums that are asked for (null: not) on one scratch block.
int run_sums(const ColumnSums* cols, const RowSums* rws, const SlopeSums* sums_in, cudaStream_t st) {
  SlopeSums sums{};
  size_t bytes = cols || rws ? sums_scratch_bytes(cols, rws) : 0;
  if (sums_in) {
    sums = *sums_in;
    Scratch sc;
    sc.take<float>(slope_sums_parts(sums.rows, sums.n) * sums.n);
    bytes = sc.used() > bytes ? sc.used() : bytes;
  }
  void* base = nullptr;
  Call call(st);
  cudaError_t e = call.scratch(bytes, &base);
  if (e == cudaSuccess && (cols || rws)) {
    Scratch sc(base);
    e = launch_sums(cols, rws, sc, st);
  }
  if (e == cudaSuccess && sums_in) {
    Scratch sc(base);
    sums.part = sc.take<float>(slope_sums_parts(sums.rows, sums.n) * sums.n);
    e = launch_slope_sums(sums, st);
  }
  return call.end(e);
}

int clip(const void* const* grads, void* const* out, const int64_t* counts, const int* dtypes, int64_t num, bool scale,
         double max_norm, float* norm, cudaStream_t st) {
  if (num < 0 || !norm || (num > 0 && (!grads || !counts || !dtypes || (scale && !out)))) return TOPK_EINVAL;
  if (scale && !(max_norm >= 0.0)) return TOPK_EINVAL;
  std::vector<ClipTensor> list(static_cast<size_t>(num));
  for (int64_t i = 0; i < num; ++i) {
    if (counts[i] < 0 || !known_dtype(dtypes[i]) || (counts[i] > 0 && (!grads[i] || (scale && !out[i])))) return TOPK_EINVAL;
    if (counts[i] > (int64_t(1) << 44)) return TOPK_EUNSUPPORTED;
    const int64_t size = static_cast<int64_t>(value_bytes(dtypes[i]));
    if (scale && grads[i] != out[i] && meet(vector(grads[i], counts[i], size), vector(out[i], counts[i], size))) return TOPK_EINVAL;
    list[static_cast<size_t>(i)] = ClipTensor{grads[i], scale ? out[i] : nullptr, counts[i], dtypes[i]};
  }
  void* base = nullptr;
  Words words;
  Call call(st);
  const cudaError_t e = call.scratch(clip_scratch_bytes(), &base, &words);
  if (e != cudaSuccess) return call.end(e);
  Scratch sc(base);
  return call.end(launch_clip(list.data(), num, scale, static_cast<float>(max_norm), norm, words, sc, st));
}

// A parameter that is one number, or one a row: numbers are checked.
bool outside(const void* rows, double v, double low, double high) { return !rows && !(v >= low && v <= high); }

int sample(const void* logits, int64_t ld, int dtype, int64_t rows, int64_t n, const float* u, double temperature,
           const float* temperatures, int64_t top_k, const int32_t* top_ks, double top_p, const float* top_ps, double min_p,
           const float* min_ps, int64_t* tokens, float* logprobs, cudaStream_t st) {
  if (!known_dtype(dtype) || rows < 0 || n < 1) return TOPK_EINVAL;
  if (outside(temperatures, temperature, 0.0, FLT_MAX) || (!top_ks && top_k < 0) || outside(top_ps, top_p, 0.0, 1.0) ||
      outside(min_ps, min_p, 0.0, 1.0))
    return TOPK_EINVAL;
  if (rows == 0) return TOPK_OK;
  if (!logits || !u || !tokens || !logprobs || ld < n) return TOPK_EINVAL;
  if (rows > kMaxExtent || n > kTokensMaxLen) return TOPK_EUNSUPPORTED;
  if (clash({vector(tokens, rows, 8), vector(logprobs, rows, 4)},
            {matrix(logits, rows, n, ld, static_cast<int64_t>(value_bytes(dtype))), vector(u, rows, 4), vector(temperatures, rows, 4),
             vector(top_ks, rows, 4), vector(top_ps, rows, 4), vector(min_ps, rows, 4)}))
    return TOPK_EINVAL;
  const float t = static_cast<float>(temperature), m = static_cast<float>(min_p);
  const TokenDraw p{logits, ld, dtype, rows, static_cast<int>(n), u, t, static_cast<float>(top_p), m, top_ks || top_k > n ? 0 : static_cast<int>(top_k), temperatures, top_ps, min_ps, top_ks,
                    tokens, logprobs, t > 0.0f ? 1.4426950408889634 / static_cast<double>(t) : 0.0, m > 0.0f ? std::log(static_cast<double>(m)) : 0.0};
  return status_of(launch_tokens(p, st));
}

// Whether rows of experts are described soundly; TOPK_OK or the error.
int check_rows(int dtype, int64_t tokens, int64_t k, int64_t d, int64_t rows) {
  if (!known_dtype(dtype) || tokens < 0 || k < 1 || d < 1 || rows < 0) return TOPK_EINVAL;
  if (tokens > kMaxExtent || k > kMaxExtent || d > (1 << 30) || rows >= (int64_t(1) << 29)) return TOPK_EUNSUPPORTED;
  return tokens * k >= (int64_t(1) << 29) ? TOPK_EUNSUPPORTED : TOPK_OK;
}

int dispatch(const Dispatch& p, cudaStream_t st) {
  if (p.experts < 1) return TOPK_EINVAL;
  if (int e = check_rows(p.dtype, p.tokens, p.k, p.d, 0)) return e;
  if (p.experts > kMostExperts) return TOPK_EUNSUPPORTED;
  if (!p.offsets) return TOPK_EINVAL;
  const int64_t size = static_cast<int64_t>(value_bytes(p.dtype)), total = p.tokens * p.k;
  if (p.tokens == 0) return status_of(cudaMemsetAsync(p.offsets, 0, sizeof(int64_t) * static_cast<size_t>(p.experts + 1), st));
  if (!p.x || p.ldx < p.d || !p.idx || !p.xs || !p.place) return TOPK_EINVAL;
  if (clash({vector(p.xs, total * p.d, size), vector(p.place, total, 8), vector(p.offsets, p.experts + 1, 8)},
            {matrix(p.x, p.tokens, p.d, p.ldx, size), vector(p.idx, total, 8)}))
    return TOPK_EINVAL;
  void* base = nullptr;
  Call call(st);
  const cudaError_t e = call.scratch(dispatch_scratch_bytes(p), &base);
  if (e != cudaSuccess) return call.end(e);
  Scratch sc(base);
  return call.end(launch_dispatch(p, sc, st));
}

int combine(const Combine& p, cudaStream_t st) {
  if (int e = check_rows(p.dtype, p.tokens, p.k, p.d, p.rows)) return e;
  if (p.tokens == 0) return TOPK_OK;
  if (!p.place || !p.y || (p.rows > 0 && (!p.ys || p.ldys < p.d))) return TOPK_EINVAL;
  const int64_t size = static_cast<int64_t>(value_bytes(p.dtype));
  if (clash({vector(p.y, p.tokens * p.d, size)}, {matrix(p.ys, p.rows, p.d, p.ldys, size), vector(p.place, p.tokens * p.k, 8),
                                                  vector(p.weights, p.tokens * p.k, size)}))
    return TOPK_EINVAL;
  return status_of(launch_combine(p, st));
}

int combine_backward(const Combine& p, cudaStream_t st) {
  if (int e = check_rows(p.dtype, p.tokens, p.k, p.d, p.rows)) return e;
  if (!p.dys && !p.dweights) return TOPK_OK;
  const int64_t size = static_cast<int64_t>(value_bytes(p.dtype)), total = p.tokens * p.k;
  if (p.tokens == 0)
    return p.dys ? status_of(cudaMemsetAsync(p.dys, 0, static_cast<size_t>(size * p.rows * p.d), st)) : TOPK_OK;
  if (!p.place || !p.dy || p.lddy < p.d || (p.dweights && p.rows > 0 && (!p.ys || p.ldys < p.d))) return TOPK_EINVAL;
  if (clash({vector(p.dys, p.rows * p.d, size), vector(p.dweights, total, size)},
            {matrix(p.dweights ? p.ys : nullptr, p.rows, p.d, p.ldys, size), matrix(p.dy, p.tokens, p.d, p.lddy, size),
             vector(p.place, total, 8), vector(p.weights, total, size)}))
    return TOPK_EINVAL;
  void* base = nullptr;
  Call call(st);
  const cudaError_t e = call.scratch(combine_backward_scratch_bytes(p), &base);
  if (e != cudaSuccess) return call.end(e);
  Scratch sc(base);
  return call.end(launch_combine_backward(p, sc, st));
}

// A cache's tensor: `row` contiguous bytes at each of batch x heads x rows places.
struct Rows4 {
  uintptr_t at;
  int64_t n[3], by[3], row;  // places and the bytes between them, by batch, head and row
  Rows4(const View& v, int64_t batch, int64_t heads, int64_t rows, int64_t dim, int64_t size)
      : at(reinterpret_cast<uintptr_t>(v.data)), n{batch, heads, rows}, by{v.batch * size, v.head * size, v.row * size}, row(dim * size) {}
  bool sound() const { return by[0] >= 0 && by[1] >= 0 && by[2] >= 0; }
  bool any() const { return at && n[0] > 0 && n[1] > 0 && n[2] > 0 && row > 0; }
  int64_t reach() const { return (n[0] - 1) * by[0] + (n[1] - 1) * by[1] + (n[2] - 1) * by[2] + row; }
  // Whether no byte belongs to two places (as far as the distances, from the smallest on, each pass what lies within).
  bool apart() const {
    int64_t within = row;
    bool used[3] = {};
    for (int step = 0; step < 3; ++step) {
      int d = -1;
      for (int i = 0; i < 3; ++i)
        if (!used[i] && n[i] > 1 && (d < 0 || by[i] < by[d])) d = i;
      if (d < 0) break;
      if (by[d] < within) return false;
      used[d] = true;
      within = (n[d] - 1) * by[d] + within;
    }
    return true;
  }
};
// Whether a row of a's and one of b's, b being `off` bytes behind, have a byte in common, by the distances order[level ... 2] (the
// largest first): a place of one against one of the other, of which the distance leaves two to try, since all that lies
// within one of its steps is shorter than it.
bool meet_at(const Rows4& a, const Rows4& b, int64_t off, const int* order, int level) {
  while (level < 3 && a.n[order[level]] < 2) ++level;
  if (level == 3) return off < a.row && -off < b.row;
  const int64_t d = a.by[order[level]], most = a.n[order[level]] - 1;
  const int64_t low = off >= 0 ? off / d : -((-off + d - 1) / d);
  for (int64_t q = low; q <= low + 1; ++q)
    if (q >= -most && q <= most && meet_at(a, b, off - q * d, order, level + 1)) return true;
  return false;
}
// Whether two have a byte in common; where they lie on different grids, whether their ranges meet.
bool meet(const Rows4& a, const Rows4& b) {
  if (!a.any() || !b.any()) return false;
  if (b.at < a.at) return meet(b, a);
  if (b.at - a.at >= static_cast<uintptr_t>(a.reach())) return false;
  for (int i = 0; i < 3; ++i)
    if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.by[i] != b.by[i])) return true;
  if (!a.apart() || !b.apart()) return true;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int x, int y) { return a.by[x] > a.by[y]; });
  return meet_at(a, b, static_cast<int64_t>(b.at - a.at), order, 0);
}
bool clash(std::initializer_list<Rows4> outs, std::initializer_list<Rows4> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Rows4& i : ins)
      if (meet(*o, i)) return true;
    for (auto p = outs.begin(); p != o; ++p)
      if (meet(*o, *p)) return true;
  }
  return false;
}
View view_of(const topk_view_t* v) { return v ? View{v->data, v->batch, v->head, v->row} : View{nullptr, 0, 0, 0}; }

int check_cache(int dtype, int weights_dtype, bool weighted, int64_t batch, int64_t heads, int64_t capacity, int64_t key_dim,
                int64_t value_dim, int64_t group, int64_t queries) {
  if (!known_dtype(dtype) || batch < 0 || heads < 1 || capacity < 1 || key_dim < 1 || value_dim < 1) return TOPK_EINVAL;
  if (weighted && (!known_dtype(weights_dtype) || group < 1 || queries < 0)) return TOPK_EINVAL;
  if (batch > kMaxExtent || heads > kMaxExtent || capacity > kMaxExtent || key_dim > kMaxExtent || value_dim > kMaxExtent ||
      (weighted && (group > kMaxExtent || queries > kMaxExtent)) || batch * heads > kMaxExtent)
    return TOPK_EUNSUPPORTED;
  // (byte counts stay below 2^63)
  const int64_t most = int64_t(1) << 40, dim = key_dim > value_dim ? key_dim : value_dim;
  if (dim > (1 << 20) || batch * heads > most / capacity || (weighted && (group * queries > (1 << 30) || group * queries > most / heads))) return TOPK_EUNSUPPORTED;
  return TOPK_OK;
}

int evict(const Evict& p, cudaStream_t st) {
  const bool weighted = p.weights.data != nullptr;
  if (int e = check_cache(p.dtype, p.weights_dtype, weighted, p.batch, p.heads, p.capacity, p.key_dim, p.value_dim, p.group, p.queries)) return e;
  if (p.keep < 1 || p.recent < 0 || p.recent > p.keep) return TOPK_EINVAL;
  if (p.keep > kMaxExtent || p.batch * p.heads > (int64_t(1) << 40) / p.keep) return TOPK_EUNSUPPORTED;
  if (p.batch == 0) return TOPK_OK;
  if (!p.keys.data || !p.values.data || !p.score.data || !p.lengths || !p.out_keys || !p.out_values || !p.out_score || !p.out_kept || !p.out_lengths)
    return TOPK_EINVAL;
  const int64_t size = static_cast<int64_t>(value_bytes(p.dtype)), rows = p.batch * p.heads;
  const Rows4 keys(p.keys, p.batch, p.heads, p.capacity, p.key_dim, size), values(p.values, p.batch, p.heads, p.capacity, p.value_dim, size);
  const Rows4 score(p.score, p.batch, p.heads, 1, p.capacity, 4);
  const Rows4 weights(p.weights, p.batch, p.heads * p.group, p.queries, weighted ? p.capacity : 0,
                      weighted ? static_cast<int64_t>(value_bytes(p.weights_dtype)) : 1);
  if (!keys.sound() || !values.sound() || !score.sound() || (weighted && !weights.sound())) return TOPK_EINVAL;
  auto flat = [](const void* at, int64_t n, int64_t bytes) { return Rows4(View{const_cast<void*>(at), 0, 0, 0}, 1, 1, 1, n, bytes); };
  if (clash({flat(p.out_keys, rows * p.keep * p.key_dim, size), flat(p.out_values, rows * p.keep * p.value_dim, size),
             flat(p.out_score, rows * p.keep, 4), flat(p.out_kept, rows * p.keep, 8), flat(p.out_lengths, p.batch, 8)},
            {keys, values, score, weights, flat(p.lengths, p.batch, 8)}))
    return TOPK_EINVAL;
  void* base = nullptr;
  Call call(st);
  const cudaError_t e = call.scratch(evict_scratch_bytes(p), &base);
  if (e != cudaSuccess) return call.end(e);
  Scratch sc(base);
  return call.end(launch_evict(p, sc, st));
}

int replace(const Replace& p, cudaStream_t st) {
  const bool weighted = p.weights.data != nullptr;
  if (int e = check_cache(p.dtype, p.weights_dtype, weighted, p.batch, p.heads, p.capacity, p.key_dim, p.value_dim, p.group, p.queries)) return e;
  if (p.recent < 0 || p.recent >= p.capacity) return TOPK_EINVAL;
  if (p.batch == 0) return TOPK_OK;
  if (!p.keys.data || !p.values.data || !p.score.data || !p.positions.data || !p.lengths || !p.key.data || !p.value.data || !p.slots) return TOPK_EINVAL;
  const int64_t size = static_cast<int64_t>(value_bytes(p.dtype));
  const Rows4 keys(p.keys, p.batch, p.heads, p.capacity, p.key_dim, size), values(p.values, p.batch, p.heads, p.capacity, p.value_dim, size);
  const Rows4 score(p.score, p.batch, p.heads, 1, p.capacity, 4), positions(p.positions, p.batch, p.heads, 1, p.capacity, 8);
  const Rows4 key(p.key, p.batch, p.heads, 1, p.key_dim, size), value(p.value, p.batch, p.heads, 1, p.value_dim, size);
  const Rows4 weights(p.weights, p.batch, p.heads * p.group, p.queries, weighted ? p.capacity : 0,
                      weighted ? static_cast<int64_t>(value_bytes(p.weights_dtype)) : 1);
  const Rows4 slots(View{p.slots, p.heads, 1, 0}, p.batch, p.heads, 1, 1, 8), lengths(View{const_cast<int64_t*>(p.lengths), 1, 0, 0}, p.batch, 1, 1, 1, 8);
  for (const Rows4* r : {&keys, &values, &score, &positions})
    if (!r->sound() || !r->apart()) return TOPK_EINVAL;
  if (!key.sound() || !value.sound() || (weighted && !weights.sound())) return TOPK_EINVAL;
  if (clash({keys, values, score, positions, slots}, {key, value, weights, lengths})) return TOPK_EINVAL;
  return status_of(launch_replace(p, st));
}

}  // namespace

cudaError_t ops_take_status(cudaStream_t st, int* status) {
  int* word = nullptr;
  StreamKey key;
  cudaError_t e = stream_key(st, &key);
  if (e != cudaSuccess) return e;
  const StreamHold hold(key);
  {
    std::lock_guard<std::mutex> lock(g_mu);
    const auto it = g_blocks.find(key);
    if (it != g_blocks.end()) word = it->second.words;
  }
  *status = kDevOk;
  if (!word) return cudaSuccess;
  e = cudaMemcpy(status, word, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && *status != kDevOk) e = cudaMemset(word, 0, sizeof(int));
  return e;
}

}  // namespace tk

using namespace tk;

extern "C" {

int topk_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, const void* residual,
                int64_t ldr, int dtype, int64_t rows, int64_t inner, int64_t outer, int act, void* y, int64_t ldy,
                void* pre, int64_t ldp, void* stream) {
  return guarded([&] {
    return linear(x, ldx, w, ldw, bias, residual, ldr, dtype, rows, inner, outer, act, y, ldy, pre, ldp,
                  static_cast<cudaStream_t>(stream));
  });
}

int topk_linear_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                         const void* pre, int64_t ldp, int dtype, int64_t rows, int64_t inner, int64_t outer, int act,
                         void* dx, void* dw, void* dbias, void* stream) {
  return guarded([&] {
    return linear_backward(dy, lddy, x, ldx, w, ldw, pre, ldp, dtype, rows, inner, outer, act, dx, dw, dbias,
                           static_cast<cudaStream_t>(stream));
  });
}

int topk_linear_backward_selected(const void* dvals, const void* vals, const int64_t* idx, int64_t count, int per_row,
                                  const void* x, int64_t ldx, const void* w, int64_t ldw, int dtype, int64_t rows,
                                  int64_t inner, int64_t outer, int act, void* dx, void* dw, void* dbias, void* stream) {
  return guarded([&]() -> int {
    if (int e = check_places(idx, count, per_row, dtype, rows, outer, inner)) return e;
    if (act != TOPK_ACT_NONE && act != TOPK_ACT_RELU) return TOPK_EINVAL;
    const Places p{idx, count, per_row != 0, rows, outer, per_row ? rows * count : count};
    if (p.total > 0 && (!dvals || (act == TOPK_ACT_RELU && !vals))) return TOPK_EINVAL;
    if ((dw && rows > 0 && (!x || ldx < inner)) || (dx && (!w || ldw < inner))) return TOPK_EINVAL;
    const int64_t size = static_cast<int64_t>(value_bytes(dtype));
    if (clash({vector(dx, rows * inner, size), vector(dw, outer * inner, size), vector(dbias, outer, size)},
              {vector(dvals, p.total, size), vector(act == TOPK_ACT_RELU ? vals : nullptr, p.total, size),
               vector(idx, p.total, sizeof(int64_t)), matrix(dw ? x : nullptr, rows, inner, ldx, size),
               matrix(dx ? w : nullptr, outer, inner, ldw, size)}))
      return TOPK_EINVAL;
    const Coef coef{dvals, act == TOPK_ACT_RELU ? vals : nullptr};
    const ColumnSums c{p, coef, dtype, x, ldx, inner, nullptr, 0, dw, dbias, nullptr};
    const RowSums r{p, coef, dtype, w, ldw, inner, nullptr, dx};
    return run_sums(dw || dbias ? &c : nullptr, dx && rows > 0 ? &r : nullptr, nullptr, static_cast<cudaStream_t>(stream));
  });
}

int topk_decode(const void* vals, const int64_t* idx, int64_t count, int per_row, const void* w, int64_t ldw,
                const void* bias, int dtype, int64_t rows, int64_t n, int64_t d, void* y, void* stream) {
  return guarded([&]() -> int {
    if (int e = check_places(idx, count, per_row, dtype, rows, n, d)) return e;
    if (rows == 0) return TOPK_OK;
    const Places p{idx, count, per_row != 0, rows, n, per_row ? rows * count : count};
    if (!y || !w || ldw < d || (p.total > 0 && !vals)) return TOPK_EINVAL;
    const int64_t size = static_cast<int64_t>(value_bytes(dtype));
    if (clash({vector(y, rows * d, size)}, {vector(vals, p.total, size), vector(idx, p.total, sizeof(int64_t)),
                                            matrix(w, n, d, ldw, size), vector(bias, d, size)}))
      return TOPK_EINVAL;
    const RowSums r{p, Coef{vals, nullptr}, dtype, w, ldw, d, bias, y};
    return run_sums(nullptr, &r, nullptr, static_cast<cudaStream_t>(stream));
  });
}

int topk_decode_backward(const void* dy, int64_t lddy, const void* vals, const int64_t* idx, int64_t count, int per_row,
                         const void* w, int64_t ldw, int dtype, int64_t rows, int64_t n, int64_t d, void* dvals,
                         void* dw, void* dbias, void* stream) {
  return guarded([&]() -> int {
    if (int e = check_places(idx, count, per_row, dtype, rows, n, d)) return e;
    const Places p{idx, count, per_row != 0, rows, n, per_row ? rows * count : count};
    if (rows > 0 && (dvals || dw || dbias) && (!dy || lddy < d)) return TOPK_EINVAL;
    if (p.total > 0 && ((dw && !vals) || (dvals && (!w || ldw < d)))) return TOPK_EINVAL;
    const int64_t size = static_cast<int64_t>(value_bytes(dtype));
    if (clash({vector(dvals, p.total, size), vector(dw, n * d, size), vector(dbias, d, size)},
              {matrix(dy, rows, d, lddy, size), vector(dw ? vals : nullptr, p.total, size), vector(idx, p.total, sizeof(int64_t)),
               matrix(dvals ? w : nullptr, n, d, ldw, size)}))
      return TOPK_EINVAL;
    if (rows == 0) {  // sums over no rows
      cudaStream_t st = static_cast<cudaStream_t>(stream);
      cudaError_t e = cudaSuccess;
      if (dw) e = cudaMemsetAsync(dw, 0, value_bytes(dtype) * static_cast<size_t>(n * d), st);
      if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, value_bytes(dtype) * static_cast<size_t>(d), st);
      if (e == cudaSuccess && dvals && p.total > 0)
        e = cudaMemsetAsync(dvals, 0, value_bytes(dtype) * static_cast<size_t>(p.total), st);
      return status_of(e);
    }
    const ColumnSums c{p, Coef{vals, nullptr}, dtype, dy, lddy, d, w, ldw, dw, nullptr, dvals};
    const SlopeSums s{dy, lddy, nullptr, 0, dtype, rows, d, kActNone, nullptr, 0, 0, dbias, nullptr};
    return run_sums(dw || dvals ? &c : nullptr, nullptr, dbias ? &s : nullptr, static_cast<cudaStream_t>(stream));
  });
}

int topk_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t num, float* norm,
                   void* stream) {
  return guarded([&] {
    return clip(grads, nullptr, counts, dtypes, num, false, 0.0, norm, static_cast<cudaStream_t>(stream));
  });
}

int topk_clip_grad_norm(const void* const* grads, void* const* out, const int64_t* counts, const int* dtypes,
                        int64_t num, double max_norm, float* norm, void* stream) {
  return guarded([&] {
    return clip(grads, out, counts, dtypes, num, true, max_norm, norm, static_cast<cudaStream_t>(stream));
  });
}

int topk_sample(const void* logits, int64_t ld, int dtype, int64_t rows, int64_t n, const float* u, double temperature,
                const float* temperatures, int64_t top_k, const int32_t* top_ks, double top_p, const float* top_ps,
                double min_p, const float* min_ps, int64_t* tokens, float* logprobs, void* stream) {
  return guarded([&] {
    return sample(logits, ld, dtype, rows, n, u, temperature, temperatures, top_k, top_ks, top_p, top_ps, min_p, min_ps, tokens,
                  logprobs, static_cast<cudaStream_t>(stream));
  });
}

int topk_dispatch(const void* x, int64_t ldx, const int64_t* idx, int dtype, int64_t tokens, int64_t k, int64_t experts,
                  int64_t d, void* xs, int64_t* place, int64_t* offsets, void* stream) {
  return guarded([&] {
    return dispatch(Dispatch{x, ldx, idx, tokens, k, experts, d, dtype, xs, place, offsets}, static_cast<cudaStream_t>(stream));
  });
}

int topk_combine(const void* ys, int64_t ldys, int64_t rows, const int64_t* place, const void* weights, int dtype,
                 int64_t tokens, int64_t k, int64_t d, void* y, void* stream) {
  return guarded([&] {
    return combine(Combine{ys, ldys, rows, place, weights, tokens, k, d, dtype, y, nullptr, 0, nullptr, nullptr},
                   static_cast<cudaStream_t>(stream));
  });
}

int topk_combine_backward(const void* dy, int64_t lddy, const void* ys, int64_t ldys, int64_t rows, const int64_t* place,
                          const void* weights, int dtype, int64_t tokens, int64_t k, int64_t d, void* dys, void* dweights,
                          void* stream) {
  return guarded([&] {
    return combine_backward(Combine{ys, ldys, rows, place, weights, tokens, k, d, dtype, nullptr, dy, lddy, dys, dweights},
                            static_cast<cudaStream_t>(stream));
  });
}

int topk_evict(const topk_view_t* keys, const topk_view_t* values, const topk_view_t* score, const int64_t* lengths,
               const topk_view_t* weights, int weights_dtype, int64_t group, int64_t queries, int dtype, int64_t batch,
               int64_t heads, int64_t capacity, int64_t key_dim, int64_t value_dim, int64_t keep, int64_t recent,
               void* out_keys, void* out_values, float* out_score, int64_t* out_kept, int64_t* out_lengths, void* stream) {
  return guarded([&] {
    return evict(Evict{view_of(keys), view_of(values), view_of(score), lengths, view_of(weights), weights_dtype, group, queries, dtype,
                       batch, heads, capacity, key_dim, value_dim, keep, recent, out_keys, out_values, out_score, out_kept, out_lengths},
                 static_cast<cudaStream_t>(stream));
  });
}

int topk_replace(const topk_view_t* keys, const topk_view_t* values, const topk_view_t* score, const topk_view_t* positions,
                 const int64_t* lengths, const topk_view_t* key, const topk_view_t* value, const topk_view_t* weights,
                 int weights_dtype, int64_t group, int64_t queries, int dtype, int64_t batch, int64_t heads,
                 int64_t capacity, int64_t key_dim, int64_t value_dim, int64_t recent, int64_t* slots, void* stream) {
  return guarded([&] {
    return replace(Replace{view_of(keys), view_of(values), view_of(score), view_of(positions), lengths, view_of(key), view_of(value),
                           view_of(weights), weights_dtype, group, queries, dtype, batch, heads, capacity, key_dim, value_dim, recent, slots},
                   static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"

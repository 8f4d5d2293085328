// C entries of the operators around the selection (declared in include/topk.h):
// argument checks, the per-(device, stream) scratch block and the launches.
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

}  // extern "C"

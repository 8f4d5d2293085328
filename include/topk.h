/*
 * topk.h -- C ABI of the GB300 Prof-K top-k selection engine (libtopk_gb300.so).
 *
 * The method is Prof-K ("Prof-K: Probabilistic One-Pass Filtering for
 * Efficient Top-k Selection", sections 3-4 and Algorithm 1): draw S uniform
 * positions, take the t-th largest sampled element as a threshold tau, stream
 * the input once keeping every element that ranks at or above tau in a buffer
 * of capacity M, then select the exact top-k of the buffer.  When fewer than k
 * elements survive, or more than M do, the engine falls back to an exact
 * selection over the whole input, so every result is exact.
 *
 * Conventions shared by every entry point:
 *   - All array pointers are DEVICE pointers owned by the caller.  x is
 *     row-major and contiguous, rows x n elements of the given dtype.
 *   - out_vals has the dtype of x and holds the input's own bits at the chosen
 *     positions; out_idx is int64.
 *   - Order: each output row lists the k winners by (value descending, index
 *     ascending) -- equal values go to the lower index, as in "Rank by
 *     Counting" (top-k task 1).  With largest == 0 the value order is reversed
 *     (smallest first) and ties still go to the lower index.  NaN ranks above
 *     every number (so it comes last when largest == 0), all NaNs are equal,
 *     -0 equals +0.
 *   - The call is asynchronous on `stream` (a cudaStream_t, NULL = legacy
 *     default stream) and does no host synchronisation, except that
 *     topk_select_ex synchronises the stream when `stats` is non-NULL.
 *   - The library keeps a per-(device, stream) workspace for the sample, the
 *     threshold, the candidate buffer and counters (and, for one selection
 *     over 16-byte aligned data with k >= 3072, or with 512 <= k < 3072 and
 *     more expected survivors than one refinement block caches, 32 MiB of
 *     bin regions into which the filter places its survivors); it grows on
 *     demand with stream-ordered allocation and is never shrunk.  Calls that
 *     share a stream are ordered, whichever threads make them (a call holds
 *     the stream's workspace until its last launch is enqueued); calls on
 *     different streams, and on the per-thread default streams of different
 *     threads, use different workspaces.
 *     A call on a stream that is being captured takes its
 *     workspace from the graph instead (allocated, and released, where it stands
 *     in it); its status is not told to topk_last_status.
 *   - Errors are returned as topk_status_t codes; nothing is thrown across the
 *     ABI and no message is printed.
 */
#ifndef TOPK_GB300_H
#define TOPK_GB300_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { TOPK_F32 = 0, TOPK_BF16 = 1 } topk_dtype_t;

typedef enum {
  TOPK_OK = 0,
  TOPK_EINVAL = -1,        /* bad argument: null pointer, k < 1, k > n, eps outside [0,1), ... */
  TOPK_ENOMEM = -2,        /* workspace allocation failed */
  TOPK_ECUDA = -3,         /* a CUDA runtime call or kernel launch failed */
  TOPK_EUNSUPPORTED = -4,  /* valid request outside the engine's limits (see topk_select) */
  TOPK_ETIMEOUT = -5       /* a bounded device-side wait gave up (with stats, or from topk_last_status) */
} topk_status_t;

/* Parameter rule for (t, M).  Both use Algorithm 1's sample size S.
 *   TOPK_RULE_EXACT (default): t and M from the exact binomial tails of the
 *     with-replacement sampler, eps/2 for recall failure and eps/2 for
 *     overflow (Theorem 3's split without the normal approximation).
 *   TOPK_RULE_ALG1: t and M as Algorithm 1 prints them (Eq. 6, Eq. 12 and
 *     the t = 1 sparse rule).  Results stay exact; only the miss rate differs. */
typedef enum { TOPK_RULE_EXACT = 0, TOPK_RULE_ALG1 = 1 } topk_rule_t;

/* Which pipeline ran (or is forced).
 *   TOPK_PATH_DIRECT: exact radix select straight over each row (small rows, or
 *     when the sample would be at least half the row).
 *   TOPK_PATH_PROFK:  sample -> threshold -> one-pass filter -> exact refine,
 *     with the full-input fallback on a miss.
 *   TOPK_PATH_EXACT:  the full-input radix select of the fallback, used for
 *     large rows when eps == 0. */
typedef enum {
  TOPK_PATH_AUTO = 0,
  TOPK_PATH_DIRECT = 1,
  TOPK_PATH_PROFK = 2,
  TOPK_PATH_EXACT = 3
} topk_path_t;

/* Tuning and test knobs.  Initialise with topk_options_init(). */
typedef struct {
  int64_t s_min;       /* Algorithm 1 S_min (default 32768) */
  int64_t s_max;       /* Algorithm 1 S_max (default 131072) */
  double cost_ratio;   /* tau_B / tau_A of Eq. 13 (default 1); 0 = as measured on this device by
                          topk_autotune (1 before that), which also applies the measured
                          Prof-K / direct crossover to the automatic path choice */
  int rule;            /* topk_rule_t (default TOPK_RULE_EXACT) */
  int path;            /* topk_path_t; TOPK_PATH_AUTO lets the engine choose */
  uint64_t seed;       /* Philox key for the sampler (default fixed) */
  int64_t counter;     /* Philox call counter; -1 = next value of a per-process counter */
  int force_miss;      /* non-zero: every row takes the fallback (fault injection on the host) */
  int64_t m_override;  /* > 0: use this buffer capacity M instead of the rule's */
  int64_t t_override;  /* > 0: use this threshold rank t instead of the rule's */
  /* Optional cudaEvent_t handles (NULL = none) recorded on `stream` at the
   * stage boundaries of the Prof-K path: [0] before the sample kernel, [1]
   * after it, [2] after the threshold selection, [3] after the filter, [4]
   * after the fallback check, [5] after the final selection.  The caller owns
   * the events; they are only recorded, never created or destroyed here. */
  void* events[6];
  /* Non-zero: the caller needs only the set of winners (BatchTopK keeps the
   * K largest activations, in any order: Prof-K paper, section 5).  For
   * selections refined on the grid (k >= 8192, at most 4 selections) the
   * k winners are then written in no particular order and the final sort
   * is skipped; every other path still sorts.  The set, the values and the
   * positions are exact either way.  Default 0. */
  int unsorted;
  /* > 0: limit in nanoseconds of each grid-wide wait of the exact fallback
   * (default 0 = 2 s).  After it the kernel records a timeout, returns, and
   * the call reports TOPK_ETIMEOUT (with stats, or from topk_last_status). */
  int64_t wait_limit_ns;
  /* Testing only (fault injection on the host's request, no GPU fault): when
   * the fallback runs, one of its blocks leaves its first grid-wide wait
   * without arriving, so every other block's bounded wait runs out.  The
   * call's output is then undefined and its status is TOPK_ETIMEOUT; the next
   * call on the stream starts clean.  Default 0. */
  int inject_wait_timeout;
  /* Relaxed recall (Prof-K paper, abstract: "relaxing the recall target (e.g.,
   * recovering 95% of the true top-k values)").  0 (default) or >= 1: exact.
   * In (0, 1): the threshold rank t is chosen for rank ceil(recall * k)
   * instead of k, so that P[fewer than ceil(recall * k) of the true top-k
   * survive] <= eps/2, and fewer than k survivors no longer take the
   * fallback: when R < k, the first R places of the row hold the exact top-R
   * (all of them true top-k elements), sorted as usual, and places R..k-1
   * hold index -1 and the value -inf (+inf when largest == 0).  A buffer
   * overflow (R > M) still takes the exact fallback.  Applies to the Prof-K
   * path; the direct and exact paths return the exact top-k. */
  double recall;
} topk_options_t;

/* Per-call report (row 0 for the per-row fields). */
typedef struct {
  int path;            /* topk_path_t that ran */
  int index_bits;      /* b of the composite key format below */
  int64_t S, t, M;     /* sample size, threshold rank, buffer capacity (0 on the direct path) */
  int64_t R;           /* row 0: elements that passed the filter (before any fallback) */
  int64_t misses;      /* rows whose filter result missed k <= R <= M and took the fallback */
  uint64_t tau;        /* row 0: composite key of the sampled threshold */
  int64_t tau_index;   /* row 0: position of the element tau was taken from */
  uint64_t seed;       /* Philox key and counter the sampler used */
  int64_t counter;
  int cluster;         /* CTAs per thread-block cluster in the final selection */
  int launches;        /* kernels this call launched on the stream */
  int64_t shortfalls;  /* rows that returned fewer than k winners (relaxed recall only) */
} topk_stats_t;

/* Parameters the engine would use for a selection of k out of n (host only). */
typedef struct {
  int path;            /* topk_path_t the automatic choice resolves to */
  int64_t S, t, M;
  double p_recall_fail;  /* P[R < k] (relaxed recall: P[R < ceil(recall*k)]) under the with-replacement sampler */
  double p_overflow;     /* P[R > M] */
} topk_plan_t;

/* Fills *opt with the defaults above. */
void topk_options_init(topk_options_t* opt);

/*
 * Per-row top-k (section 3: "for batched inputs ... applied in parallel to each
 * batch element").  For each of `rows` rows of n elements, writes the k
 * winners to out_vals[r*k + j] and their row-local positions to
 * out_idx[r*k + j].  eps in [0, 1) is the target probability that a row takes
 * the fallback (Theorem 3); eps == 0 selects exactly without sampling.  The
 * result never depends on eps or on the sampler.
 *   Limits: n < 2^31; k <= 188416 (EUNSUPPORTED beyond); rows == 0 is a no-op.
 *   EINVAL: null pointer (with rows > 0), rows < 0, n < 1, k < 1, k > n,
 *           eps outside [0, 1), unknown dtype.
 */
int topk_select(const void* x, int dtype, int64_t rows, int64_t n, int64_t k, int largest,
                double eps, void* out_vals, int64_t* out_idx, void* stream);

/*
 * Batch-global top-k (BatchTopK, section 5: the B x d_dict activations are
 * flattened into one vector of N = B*d_dict and the K = B*k largest are kept).
 * Treats the rows*n elements as one vector: out_vals[j], out_idx_flat[j] for
 * j < k, with flat positions r*n + c.
 *   Limits: rows*n <= 2^32 for F32 and <= 2^48 for BF16; k <= 188416.
 *   EINVAL as topk_select, with k > rows*n in place of k > n.
 */
int topk_select_global(const void* x, int dtype, int64_t rows, int64_t n, int64_t k, int largest,
                       double eps, void* out_vals, int64_t* out_idx_flat, void* stream);

/*
 * topk_select (global == 0) or topk_select_global (global != 0) with options
 * (NULL = defaults) and an optional report.  When stats is non-NULL the call
 * synchronises `stream` before returning and can return TOPK_ETIMEOUT.
 */
int topk_select_ex(const void* x, int dtype, int64_t rows, int64_t n, int64_t k, int largest,
                   double eps, void* out_vals, int64_t* out_idx, void* stream, int global,
                   const topk_options_t* opt, topk_stats_t* stats);

/* Host-only: the path and (S, t, M) the engine uses for one selection of k out
 * of n elements (n = rows*n for the global variant).  Algorithm 1 and the rule
 * in opt (NULL = defaults).  EINVAL on bad arguments. */
int topk_plan(int64_t n, int64_t k, double eps, const topk_options_t* opt, topk_plan_t* plan);

/*
 * Device-side status of the most recent selection issued on `stream` (of the
 * current device) by topk_select, topk_select_global, topk_select_ex or
 * topk_select_noalloc.  Synchronises `stream` first.  Returns TOPK_OK, or
 * TOPK_ETIMEOUT when one of that call's bounded device waits gave up (its
 * output is then undefined), or TOPK_ECUDA when its kernels found their state
 * inconsistent; CUDA errors of the synchronisation itself map to TOPK_ECUDA.
 * The status words are reset by each call, so this reports the last call
 * only.  The short-row direct path (rows of at most 32768 elements, k <= 1024)
 * keeps a status word only when topk_select_ex is given `stats`; otherwise
 * this returns TOPK_OK for it.  Calls without any selection on `stream`
 * return TOPK_OK.  TOPK_ETIMEOUT is also returned, once, when a bounded device
 * wait of topk_linear or topk_linear_backward gave up on this stream since the
 * last call of this function.
 */
int topk_last_status(void* stream);

/* Measured cost model of this device (Prof-K paper, section 4, "Optimal
 * Sample Size": the ratio tau_B / tau_A "may be estimated by lightweight
 * microbenchmarking"; Figure 3 for the crossover with a direct method). */
typedef struct {
  double tau_a_ns;      /* sampling and threshold: device time per additional sampled element */
  double tau_b_ns;      /* refinement: device time per additional buffered element, per log2 k */
  double cost_ratio;    /* tau_b_ns / tau_a_ns, the ratio of Eq. 13 and 14 */
  int64_t crossover_n;  /* smallest measured row length from which Prof-K beat the direct path
                           at every larger measured length (0: it never did) */
  int64_t crossover_k;  /* the k the crossover was measured at */
} topk_tuning_t;

/*
 * Measures the cost model on the current device with synthetic uniform f32
 * rows through the selection pipeline itself (CUDA events at its stage
 * boundaries, medians of repeated calls): tau_A from the sampling and
 * threshold stage at S = 32768 and S = 131072; tau_B from the refinement at
 * two survivor counts (k = 1024); the crossover from full selections of k out
 * of n = 2^16 ... 2^24 by the direct path and by Prof-K (eps = 1e-3).  Allocates
 * about 256 MiB of device memory for the duration and synchronises `stream`;
 * takes on the order of a second.  The result is kept for the device and used
 * by calls whose options set cost_ratio = 0.  k: the k of the crossover (0 =
 * 1024).  Errors: TOPK_EINVAL for a null `out` or k outside [0, 65536],
 * TOPK_ENOMEM / TOPK_ECUDA.
 */
int topk_autotune(int64_t k, void* stream, topk_tuning_t* out);

/* The measured cost model of the current device (TOPK_EINVAL when topk_autotune
 * has not run on it). */
int topk_tuning(topk_tuning_t* out);

/* Static text for a status code. */
const char* topk_status_str(int status);

/* Library version: major*10000 + minor*100 + patch.  0.2.0 (200) added the
 * `unsorted` field at the end of topk_options_t; 0.3.0 (300) added
 * `wait_limit_ns`, `inject_wait_timeout` and `recall` after it, `shortfalls`
 * at the end of topk_stats_t, topk_last_status, topk_autotune and topk_tuning
 * (cost_ratio = 0 meaning "measured"); 0.4.0 (400) added the operators
 * around the selection; 0.5.0 (500) those of a language model at the end of
 * this header.
 * Fill the struct with topk_options_init from the same version's library. */
int topk_version(void);

/* ------------------------------------------------------------------------
 * Stage entry points: the individual steps of the Prof-K pipeline, for tests
 * and for callers that want the pieces.
 *
 * Composite key format.  Every element is identified by a 64-bit key whose
 * unsigned order is the selection order:
 *     key = (v << b) | (2^b - 1 - i)
 * where i is the element's position in its selection (row-local, or flat for
 * the global variant), b = topk_index_bits(length of the selection), and v is
 * the order-preserving image of the value: for F32 bits u (BF16 likewise on 16
 * bits), NaN -> all ones, -0 -> +0, then v = u | signbit if u is non-negative,
 * else ~u; with largest == 0, v is complemented.  Larger key = better rank;
 * keys are distinct, so "ranks at or above tau" is simply key >= tau.
 * ------------------------------------------------------------------------ */

/* b for a selection over `len` elements: the bits needed for positions 0..len-1 (at least 1). */
int topk_index_bits(int64_t len);

/*
 * Stage 1 (section 3, sampling): for each selection r, draws S positions with
 * Philox4x32-10 -- draw j uses counter (j/2, r, counter_lo, counter_hi) and key
 * (seed_lo, seed_hi); the even draw takes the 64-bit word (w1<<32 | w0), the
 * odd one (w3<<32 | w2); the position is floor(word * len / 2^64) -- and writes
 * the composite keys of the drawn elements to out_keys[r*S + j].
 * global != 0 treats x as one selection of rows*n elements.
 */
int topk_prof_sample(const void* x, int dtype, int64_t rows, int64_t n, int global, int largest,
                     int64_t S, uint64_t seed, int64_t counter, uint64_t* out_keys, void* stream);

/*
 * Stage 3 (section 3, filtering): for each selection r, streams its elements
 * once and appends the composite key of every element with key >= tau[r] to
 * buf[r*M ...]; counts[r] receives the number R of such elements (it keeps
 * counting past M; only the first M found are stored, in no particular order).
 * tau (device, one key per selection) uses the key format above.
 */
int topk_prof_filter(const void* x, int dtype, int64_t rows, int64_t n, int global, int largest,
                     const uint64_t* tau, int64_t M, uint64_t* buf, uint64_t* counts,
                     void* stream);

/*
 * topk_select_noalloc -- the selection of topk_select (global == 0) or
 * topk_select_global (global != 0) without any device allocation.  The paper
 * has no counterpart of this entry point.
 *
 * For callers that cannot allocate while they run: a process whose device
 * memory belongs to another allocator (a framework caching allocator holding
 * nearly all of HBM, where a hidden cudaMalloc can fail or fragment it), or
 * latency-critical loops that cannot take cudaMalloc's implicit device
 * synchronisation.  All scratch comes from one static device array of 8 MiB
 * inside the library, held by every GPU that loads the library until exit.
 * The selection runs through the same kernels and the same choices of path
 * as topk_select; only the scratch memory differs.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.
 *   - Every call on a device shares the array and it keeps the last call's
 *     contents; the library clears the words that must start at zero.  Calls
 *     that overlap on the GPU (e.g. unordered streams of one device) race on
 *     the array: order them on one stream.
 *   - A request whose scratch would exceed 8 MiB returns TOPK_EUNSUPPORTED
 *     before anything is launched; use topk_select then.  About 2.2 MiB is a
 *     fixed part; the rest grows with the selections: roughly 8 bytes per
 *     sample (S) and per buffer slot (M), 16 bytes per winner (k), and 1 byte
 *     per 1024 input elements.  The 4096 x 65536 bf16 BatchTopK selection
 *     (K = 131072) fits.
 *   - A bounded device wait that gives up is reported by topk_last_status on
 *     the same stream (this call itself does not synchronise).
 * Arguments, outputs, limits and the other error codes are those of
 * topk_select / topk_select_global.
 */
int topk_select_noalloc(const void* x, int dtype, int64_t rows, int64_t n, int64_t k, int largest,
                        double eps, void* out_vals, int64_t* out_idx, int global, void* stream);

/* ------------------------------------------------------------------------
 * Operators around the selection: what a sparse autoencoder's training step
 * runs before and after topk_select_global (or topk_select, which keeps k
 * features a row) -- the encoder, the reconstruction from the selected
 * activations, their gradients, and the gradient norm with clipping.
 *
 *   - All tensors of one call have one dtype (F32 or BF16).  Matrices are
 *     row-major with unit stride along a row; ld* is the distance between
 *     rows in elements (at least the row's length).  Outputs without an ld
 *     are contiguous.  No alignment is needed beyond the element's own (rows
 *     that start on 16-byte boundaries are read faster).
 *   - Products, sums, activations and norms are formed in f32 or wider; each
 *     result is rounded once, to nearest even.  Results do not depend on the
 *     order in which blocks run: the same call gives the same bits.
 *   - Outputs marked "nullable" are not computed when null.
 *   - Outputs overlap neither inputs nor each other (EINVAL; views of one
 *     buffer may lie between each other when their rows are equally far apart),
 *     except where an entry point says so.
 *   - Extents are below 2^31 and a selection's places below 2^29 (EUNSUPPORTED
 *     beyond, and where a launch cannot count its blocks).
 *   - Scratch memory comes from a per-(device, stream) block of these
 *     operators, apart from the selection's workspace but grown and held like
 *     it.  A call on a stream that is being captured takes its scratch from the
 *     graph instead (allocated, and released, where it stands in it), so that
 *     graphs may be replayed on any stream, beside other calls.  A device wait
 *     that gives up in a replay is told to topk_last_status of the stream that
 *     was captured if topk_linear, topk_linear_backward or a norm ran on it
 *     before that; otherwise it is not told.
 * ------------------------------------------------------------------------ */

/* z, max(z, 0), z Phi(z) with the normal distribution function Phi, z / (1 + e^-z). */
typedef enum { TOPK_ACT_NONE = 0, TOPK_ACT_RELU = 1, TOPK_ACT_GELU = 2, TOPK_ACT_SILU = 3 } topk_act_t;

/*
 * y = act(x w^T + bias) + residual: x is rows x inner, w is outer x inner, y
 * rows x outer.  bias (outer values) and residual (rows x outer) are nullable;
 * residual may be y itself.  pre (nullable): x w^T + bias, kept for
 * topk_linear_backward.  rows == 0 is a no-op.
 */
int topk_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, const void* residual,
                int64_t ldr, int dtype, int64_t rows, int64_t inner, int64_t outer, int act, void* y, int64_t ldy,
                void* pre, int64_t ldp, void* stream);

/*
 * Gradients of topk_linear from dy (rows x outer), with dz = dy act'(pre):
 * dx = dz w, dw = dz^T x, dbias = the column sums of dz (each nullable; the
 * residual's gradient is dy itself).  pre is read unless act is NONE; for RELU
 * the layer's own output serves when it had no residual (the signs agree).
 * BF16 with GELU or SILU: dz enters the two products with 16 bits (of its
 * rounding to BF16 and of what that left; BF16's own 8 where x or w holds a
 * value that is not finite); dbias sums it in f32.  x is needed for dw only
 * and w for dx only.
 */
int topk_linear_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                         const void* pre, int64_t ldp, int dtype, int64_t rows, int64_t inner, int64_t outer, int act,
                         void* dx, void* dw, void* dbias, void* stream);

/*
 * A selection's places, as the entry points below take them: `idx` as
 * topk_select_global writes it (per_row == 0: `count` flat positions r*n + c)
 * or as topk_select does (per_row != 0: `count` row-local positions for each
 * row), in any order.  A position out of range (the -1 of a relaxed recall's
 * shortfall) holds no place: it adds nothing, and its gradient is 0.  A place
 * listed twice counts twice.
 */

/*
 * Gradients of topk_linear when only selected outputs carry one: dvals[s] at
 * place s, vals[s] the selected output.  With dz_s = dvals[s] act'(vals[s])
 * (act NONE or RELU): dx[r] = sum of dz_s w[c_s] over the places of row r
 * (rows x inner), dw[c] = sum of dz_s x[r_s] over those of column c (outer x
 * inner), dbias[c] = sum of dz_s; each nullable.
 */
int topk_linear_backward_selected(const void* dvals, const void* vals, const int64_t* idx, int64_t count, int per_row,
                                  const void* x, int64_t ldx, const void* w, int64_t ldw, int dtype, int64_t rows,
                                  int64_t inner, int64_t outer, int act, void* dx, void* dw, void* dbias, void* stream);

/*
 * Reconstruction from a selection out of rows x n activations: y[r] = bias +
 * the sum of vals[s] w[c_s] over the places of row r.  w is n x d (one row a
 * feature), y rows x d; bias (d values) is nullable.
 */
int topk_decode(const void* vals, const int64_t* idx, int64_t count, int per_row, const void* w, int64_t ldw,
                const void* bias, int dtype, int64_t rows, int64_t n, int64_t d, void* y, void* stream);

/*
 * Gradients of topk_decode from dy (rows x d): dvals[s] = dy[r_s] . w[c_s],
 * dw[c] = the sum of vals[s] dy[r_s] over the places of column c (n x d, zero
 * for features that were not selected), dbias = the column sums of dy; each
 * nullable.
 */
int topk_decode_backward(const void* dy, int64_t lddy, const void* vals, const int64_t* idx, int64_t count, int per_row,
                         const void* w, int64_t ldw, int dtype, int64_t rows, int64_t n, int64_t d, void* dvals,
                         void* dw, void* dbias, void* stream);

/*
 * The norm of `num` tensors taken as one vector, *norm = sqrt(sum of squares)
 * (f32, on the device; any finite input whose norm is below the f32 range's
 * end gives a finite norm).  grads, counts and dtypes are HOST arrays: device
 * pointers, elements (0 allowed) and dtypes (which may differ) of each tensor.
 */
int topk_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t num, float* norm,
                   void* stream);

/*
 * The same norm, and out[i] = grads[i] * min(1, max_norm / (*norm + 1e-6)).
 * out[i] == grads[i] clips in place; otherwise the two do not overlap.  A
 * tensor is listed once.  A norm
 * that is not finite carries over to the results as the formula says.
 * EINVAL: max_norm < 0 or NaN.
 */
int topk_clip_grad_norm(const void* const* grads, void* const* out, const int64_t* counts, const int* dtypes,
                        int64_t num, double max_norm, float* norm, void* stream);

/* ------------------------------------------------------------------------
 * Operators of a language model around the selection: the next token out of
 * its logits, tokens sorted by the experts they were routed to and back, and
 * the positions of a key-value cache that stay.  What is said of the operators
 * above (layout, rounding, overlap, scratch, capture) holds for these too.
 * ------------------------------------------------------------------------ */

/*
 * A token of each row of logits (rows x n), drawn with the number u[r] of
 * [0, 1).  Tokens stand in the selection's order (logit descending, index
 * ascending); with z = (logit - the row's largest) / temperature a token
 * weighs e^z.  Kept are
 *   the tokens that weigh at least min_p (the largest weighs 1),
 *   of those the first top_k (0: all),
 *   of those the shortest prefix whose weights sum to top_p of theirs or more,
 * at least one in each case; tokens[r] is the first in order at which the sum
 * of the weights passes u[r] times that of all kept, and logprobs[r] the
 * logarithm of its share of that.  A temperature of 0 takes the largest logit.
 * NaN and -inf are never drawn; a row of nothing else gives -1 and -inf.
 * Where a logit is +inf, only such are drawn.
 *   Weights are formed to 30 bits and added up as whole numbers, the largest as
 * 2^45 (what is less than 1 is dropped, from each of the up to some thousand
 * largest tokens and from the others' sum), so the token is that of 64-bit
 * arithmetic unless u[r] (or a filter's border) is within about 2^-29 of the edge
 * between two; weights below 2^-48 of the largest count as 0.  logprobs are off by
 * at most 2^-22 of themselves and 2^-28.
 *   Each of temperature, top_k, top_p and min_p is a number, or one a row
 * (device, `rows` values) where its pointer is not null, the number then
 * being ignored; numbers are rounded to f32.  A row's temperature that is not
 * above 0 (NaN too) takes the largest logit, its top_k below 1 keeps all, its
 * top_p and min_p outside [0, 1] count as the nearer end, or as unset where NaN.
 *   Limits: n <= 262144 (EUNSUPPORTED beyond); rows == 0 is a no-op.
 *   EINVAL: a number that is negative, NaN or infinite, top_p or min_p above 1.
 */
int topk_sample(const void* logits, int64_t ld, int dtype, int64_t rows, int64_t n, const float* u, double temperature,
                const float* temperatures, int64_t top_k, const int32_t* top_ks, double top_p, const float* top_ps,
                double min_p, const float* min_ps, int64_t* tokens, float* logprobs, void* stream);

/*
 * Rows sorted by expert.  idx (tokens x k, as topk_select writes it: an expert
 * of 0 ... experts - 1 for each token and choice) sends token t's row of x
 * (tokens x d) to k experts.  xs (tokens k rows of d, contiguous) holds the
 * rows of expert 0 first, then those of expert 1, ..., each expert's in the
 * order of t k + j; place[t k + j] is the row's number in xs; expert e has
 * rows offsets[e] to offsets[e + 1] - 1 (experts + 1 values).  A choice out of
 * range (-1 where a token was dropped) has place -1; the rows of xs that are
 * left over, at its end, are zeros.
 *   The gradient of x is topk_combine of xs's, without weights.
 *   Limits: experts <= 4096, tokens k < 2^29, d <= 2^30 (EUNSUPPORTED beyond; for
 * the way back, rows < 2^29 too).
 */
int topk_dispatch(const void* x, int64_t ldx, const int64_t* idx, int dtype, int64_t tokens, int64_t k, int64_t experts,
                  int64_t d, void* xs, int64_t* place, int64_t* offsets, void* stream);

/*
 * The way back: y[t] = the sum over j of weights[t k + j] ys[place[t k + j]]
 * (ys: rows x d, weights: tokens x k of the same dtype, nullable: all 1; y:
 * tokens x d).  A place out of range adds nothing.
 */
int topk_combine(const void* ys, int64_t ldys, int64_t rows, const int64_t* place, const void* weights, int dtype,
                 int64_t tokens, int64_t k, int64_t d, void* y, void* stream);

/*
 * Gradients of topk_combine from dy (tokens x d): dys[r] = the sum of
 * weights[t k + j] dy[t] over the places that are r (rows x d; zeros where
 * none is), dweights[t k + j] = dy[t] . ys[place[t k + j]] (0 where the place
 * is out of range); each nullable.  ys is needed for dweights only.  Rows that
 * topk_dispatch placed are each listed once; a row that is listed more often
 * is summed in the order of its places.  From 129 places on a row that takes a
 * scan over all places, for each such row and each 256 16-byte pieces of it
 * (256 values where rows are not on 16-byte boundaries).
 */
int topk_combine_backward(const void* dy, int64_t lddy, const void* ys, int64_t ldys, int64_t rows, const int64_t* place,
                          const void* weights, int dtype, int64_t tokens, int64_t k, int64_t d, void* dys, void* dweights,
                          void* stream);

/* A tensor of batch x heads x rows rows of contiguous values: distances between them, in elements (0 or more). */
typedef struct {
  void* data;
  int64_t batch, head, row;
} topk_view_t;

/*
 * What stays in a key-value cache that is cut down to `keep` positions: the
 * last `recent` ones of each sequence and, of the others, those with the
 * largest scores (NaN above all numbers, equal ones by position).
 *   keys, values: batch x heads x capacity rows of key_dim and value_dim
 *     values of `dtype`, of which the first lengths[b] positions hold tokens
 *     (device, int64; below 0 counts as 0, above the capacity as that).
 *   score: f32, batch x heads rows of capacity values (its `row` is not used):
 *     the attention weight that each position has had.
 *   weights (NULL: none): what is added to it first, batch x (heads group) x
 *     queries rows of capacity values of weights_dtype; query heads h group
 *     ... h group + group - 1 read head h.  A weight that is NaN (a query
 *     whose mask left nothing) counts as 0; behind lengths[b] none is read for
 *     its value.  The sum is rounded to f32 once and off by at most (rows + 32)
 *     2^-45 of the magnitudes' sum before that, with group queries rows; score
 *     is not changed.
 * Contiguous results: out_keys and out_values, the rows of what stays, in the
 * order of their positions (batch x heads x keep rows); out_score their score;
 * out_kept their positions; out_lengths[b] = min(lengths[b], keep).  Behind
 * that, rows and scores are zeros and positions -1.
 *   Limits: batch heads capacity and batch heads keep <= 2^40, dims <= 2^20,
 * group queries <= 2^30 (EUNSUPPORTED beyond).  EINVAL: keep < 1, recent outside [0, keep].
 */
int topk_evict(const topk_view_t* keys, const topk_view_t* values, const topk_view_t* score, const int64_t* lengths,
               const topk_view_t* weights, int weights_dtype, int64_t group, int64_t queries, int dtype, int64_t batch,
               int64_t heads, int64_t capacity, int64_t key_dim, int64_t value_dim, int64_t keep, int64_t recent,
               void* out_keys, void* out_values, float* out_score, int64_t* out_kept, int64_t* out_lengths, void* stream);

/*
 * The single-token form, in place: a new token's key and value (batch x heads
 * rows; their `row` is not used) go into each head's cache of `capacity`
 * slots.  lengths[b] is the number of tokens before it, and its position.
 * weights (as above, by slot) are added to the scores of the slots in use
 * first.  While there are fewer tokens than slots, the token takes slot
 * lengths[b]; then, the slot with the least score (NaN above all numbers,
 * equal ones: the lowest slot) of those whose position is below lengths[b] -
 * recent.  The slot's score becomes 0 and its position lengths[b]; slots[b
 * heads + h] is the slot, or -1 where every position is recent (nothing is
 * stored then).  positions: int64, batch x heads rows of capacity values.
 *   EINVAL: recent outside [0, capacity - 1].
 */
int topk_replace(const topk_view_t* keys, const topk_view_t* values, const topk_view_t* score, const topk_view_t* positions,
                 const int64_t* lengths, const topk_view_t* key, const topk_view_t* value, const topk_view_t* weights,
                 int weights_dtype, int64_t group, int64_t queries, int dtype, int64_t batch, int64_t heads,
                 int64_t capacity, int64_t key_dim, int64_t value_dim, int64_t recent, int64_t* slots, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TOPK_GB300_H */

/*
 * topk_ef.h -- C ABI of the B200 Top-k + error-feedback sparsifier and the
 * gTop-k merge of sparse (index, value) sets.
 *
 * What the calls compute (sources are web pages, cited by title and section):
 *
 *  - One error-feedback step ("Sparsified SGD with Memory", abstract: send the
 *    top-k entries and keep the accumulated error in memory; "The Convergence
 *    of Sparsified Gradient Methods", abstract: transmit a subset by
 *    magnitude, accumulate the rest locally):
 *        acc[i]      = fmaf(lr, grad[i], residual[i])      (one fp32 rounding)
 *        S           = the k indices of largest |acc|, ties to the lower index
 *        out         = (i, acc[i]) for i in S, ascending i
 *        residual[i] = +0.0f for i in S, acc[i] otherwise
 *    |x| order is the order of bits(x) & 0x7FFFFFFF as an unsigned integer
 *    (-0 == +0; NaN above +Inf).
 *
 *  - The gTop-k merge ("A Distributed Synchronous SGD Algorithm with Global
 *    Top-k Sparsification for Low Bandwidth Networks", ABSTRACT: the global
 *    top-k largest absolute values from P workers; method section: a
 *    tournament in O(log P) rounds).  Round r = 0, 1, ... while 2^r < P: every
 *    worker i that is a multiple of 2^(r+1) with i + 2^r < P replaces its set
 *    by the top min(k, |U|) of U = S_i (+) S_{i+2^r}, the union with one fp32
 *    add (round to nearest even) at common indices.  A worker without a
 *    partner in a round keeps its set.  The result is the top min(k, |S_0|)
 *    of S_0, ascending index.
 *
 * Conventions shared by every call:
 *  - Pointers marked "device" are CUDA device pointers on the current device;
 *    pointers marked "host" are host memory read before the call returns.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *    compute call is asynchronous on that stream and returns once its work
 *    is enqueued.
 *  - The caller owns every buffer, including the workspace `ws`
 *    (device memory, at least the size the matching *_workspace_bytes call
 *    returns, 256-byte aligned).  Calls on the same workspace must be ordered
 *    (same stream, or synchronised); the library allocates no memory and
 *    keeps nothing between calls except inside `ws`.  A workspace needs no
 *    initialisation: its contents before the first call (zeros, garbage, a
 *    workspace last used with other sizes) never change a result.
 *  - fp32 arrays must be 4-byte aligned; 16-byte aligned grad/residual take
 *    the vectorised path, other alignments a scalar path with identical
 *    results.
 *  - Results are deterministic and bit-identical from run to run.
 *
 * Return codes.  The return value covers argument checks and launch errors;
 * problems found on the device (a bounded wait that gave up, malformed merge
 * input) are recorded in the workspace and read back with
 * topk_ef_last_device_status().  No call traps, asserts on the device or
 * waits without bound.
 */
#ifndef TOPK_EF_H
#define TOPK_EF_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TOPK_EF_OK 0
/* null pointer, n < 0, k < 0, k > n, n > 2^31 - 1, T < 1, P < 1, k_in > n,
   offsets not starting at 0 or decreasing, misaligned fp32 pointer */
#define TOPK_EF_ERR_INVALID_ARG (-1)
/* ws_bytes smaller than the matching *_workspace_bytes() */
#define TOPK_EF_ERR_WORKSPACE (-2)
/* a CUDA launch or runtime call failed; topk_ef_last_cuda_error() has it */
#define TOPK_EF_ERR_CUDA (-3)
/* device: a bounded spin-wait gave up (outputs are undefined) */
#define TOPK_EF_ERR_DEVICE_TIMEOUT (-4)
/* device: merge input rows not strictly ascending or indices outside [0, n),
   embedding, token or teacher ids outside [0, V) */
#define TOPK_EF_ERR_BAD_INPUT (-5)
/* device: an internal count did not add up (outputs are undefined) */
#define TOPK_EF_ERR_INTERNAL (-6)

/* ---------------------------------------------------------------- compress */

/* Workspace bytes for topk_ef_compress on n elements with k kept.
   Returns 0 for invalid (n, k). */
size_t topk_ef_workspace_bytes(int64_t n, int64_t k);

/*
 * One error-feedback step on a flat fp32 tensor.
 *   grad      device, fp32[n], read only; must not overlap residual or outputs
 *   residual  device, fp32[n]; in: the memory, out: acc with the k sent slots
 *             set to +0.0f
 *   n         0 <= n <= 2^31 - 1 (indices are int32)
 *   lr        scale applied to grad inside the single fmaf
 *   k         0 <= k <= n
 *   out_idx   device, int32[k], ascending indices of the sent entries
 *   out_val   device, fp32[k], acc at those indices (signed)
 *   ws        device workspace of ws_bytes >= topk_ef_workspace_bytes(n, k)
 *
 * The compress keeps, in `ws`, the threshold of the previous call made with
 * the same residual pointer, n, k and lr ("Sparsified SGD with Memory",
 * abstract: the memory carries over from step to step, and so does the
 * magnitude of what is sent): a prefilter only, the result is exact whatever
 * it holds.  A tensor small enough for one wave of blocks (n <= 148 * 16,384
 * on a 148-SM device) takes one kernel launch; its workspace holds 8 n bytes
 * of candidate lists besides.  The launch's parameters are the same from
 * call to call apart from a host-issued call number, and the kernel keeps
 * its own call counter in `ws`, so a call captured in a CUDA graph may be
 * replayed.
 */
int topk_ef_compress(const float* grad, float* residual, int64_t n, float lr,
                     int64_t k, int32_t* out_idx, float* out_val, void* ws,
                     size_t ws_bytes, void* stream);

/*
 * topk_ef_compress_static: the same error-feedback step as topk_ef_compress,
 * for callers that cannot allocate device memory, and so cannot provide the
 * workspace: for instance code that runs inside a host program whose
 * framework owns all device memory and forbids other allocations, or a
 * latency-critical path where a cudaMalloc (which can synchronise the device)
 * is not acceptable.  The pages have no counterpart of this entry point.
 *
 * The scratch it uses in place of `ws` is a fixed array of
 * TOPK_EF_STATIC_SCRATCH_BYTES (32 MiB) inside the library's device module:
 * every GPU on which the library is used holds it until the process exits.
 * It allocates nothing itself: no cudaMalloc, cudaFree or allocating library
 * routine.  The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and keeps it; make that
 * first call before any stream capture.  Sizes whose workspace
 * (topk_ef_workspace_bytes(n, k)) exceeds the array are rejected with
 * TOPK_EF_ERR_WORKSPACE (32 MiB holds, e.g., n = 25.6M at k = 1% or
 * n = 150M at k = 0.1%).  All calls share the one array and each call resets
 * the state it needs at its start, so it keeps no result between calls; two
 * calls whose GPU work overlaps (different streams, or different host threads
 * without ordering) race on it and must not be issued.
 *   Arguments and results: exactly those of topk_ef_compress, without ws and
 *   ws_bytes.
 */
#define TOPK_EF_STATIC_SCRATCH_BYTES ((size_t)32 << 20)
int topk_ef_compress_static(const float* grad, float* residual, int64_t n, float lr,
                            int64_t k, int32_t* out_idx, float* out_val,
                            void* stream);

/*
 * Device-side status of the last topk_ef_compress_static call on the current
 * device, the counterpart of topk_ef_last_device_status(ws, stream) for the
 * library's scratch array (which the caller has no address of): synchronises
 * `stream` and returns TOPK_EF_OK, TOPK_EF_ERR_DEVICE_TIMEOUT or
 * TOPK_EF_ERR_INTERNAL (TOPK_EF_ERR_CUDA if the read-back failed).  Check it
 * before using the outputs of a call that may have hit a bounded wait.  The
 * device address of the array is looked up once per device and kept; after
 * cudaDeviceReset it is stale (as is every other device pointer of the
 * process), and neither call may be used again.
 */
int topk_ef_static_last_device_status(void* stream);

/* ------------------------------------------------------- hard threshold */

/* Workspace bytes for topk_ef_threshold on n elements; 0 for invalid n. */
size_t topk_ef_threshold_workspace_bytes(int64_t n);

/*
 * One error-feedback step of the hard-threshold sparsifier ("Rethinking
 * gradient sparsification as total error minimization", abstract: the
 * variant of Top-k whose k is set by a constant hard threshold, analysed
 * under error feedback):
 *     acc = fmaf(lr, grad, residual);
 *     the entries with key(acc) >= key(threshold) pass (|acc| at least
 *     |threshold|; NaN above +Inf, as in topk_ef_compress; a NaN threshold
 *     passes only NaNs);
 *     the first min(count, max_out) passing entries in ascending index order
 *     are sent; the others stay in memory.
 *   grad, residual, n, lr  as in topk_ef_compress
 *   threshold  compared by magnitude (its sign is ignored)
 *   max_out    >= 0: capacity of out_idx / out_val
 *   out_idx    device, int32[max_out]: ascending indices of the sent entries;
 *              slots from min(count, max_out) on are not written
 *   out_val    device, fp32[max_out]: acc at those indices
 *   out_count  device, int64 (8-byte aligned): count, the number of entries
 *              that passed (may exceed max_out)
 *   ws         device workspace of >= topk_ef_threshold_workspace_bytes(n)
 * Errors: TOPK_EF_ERR_INVALID_ARG (n out of range, max_out < 0, null or
 * misaligned pointers), TOPK_EF_ERR_WORKSPACE, TOPK_EF_ERR_CUDA.
 */
int topk_ef_threshold(const float* grad, float* residual, int64_t n, float lr,
                      float threshold, int64_t max_out, int32_t* out_idx,
                      float* out_val, int64_t* out_count, void* ws,
                      size_t ws_bytes, void* stream);

/* Workspace bytes for topk_ef_compress_batched with the same (offsets, k, T).
   offsets and k are host arrays.  Returns 0 for invalid arguments. */
size_t topk_ef_batched_workspace_bytes(const int64_t* offsets,
                                       const int64_t* k, int32_t T);

/*
 * One error-feedback step on each of T tensors stored back to back in one
 * flat bucket (per-tensor k; the tensors are independent problems).
 *   grad, residual  device, fp32[offsets[T]]; tensor l is
 *                   [offsets[l], offsets[l+1]); residual updated in place
 *   offsets         host, int64[T+1], offsets[0] = 0, non-decreasing,
 *                   offsets[T] <= 2^31 - 1
 *   k               host, int64[T], 0 <= k[l] <= offsets[l+1] - offsets[l]
 *   T               number of tensors, >= 1
 *   out_idx         device, int32[sum k]; tensor l's entries start at
 *                   sum_{j<l} k[j] and hold indices LOCAL to tensor l,
 *                   ascending
 *   out_val         device, fp32[sum k], matching acc values
 *   ws              device workspace of ws_bytes >=
 *                   topk_ef_batched_workspace_bytes(offsets, k, T)
 */
int topk_ef_compress_batched(const float* grad, float* residual,
                             const int64_t* offsets, const int64_t* k,
                             int32_t T, float lr, int32_t* out_idx,
                             float* out_val, void* ws, size_t ws_bytes,
                             void* stream);

/* ------------------------------------------------------------------ merge */

/* Workspace bytes for gtopk_merge with P sets of k_in entries keeping k.
   Returns 0 for invalid arguments. */
size_t gtopk_merge_workspace_bytes(int32_t P, int64_t k_in, int64_t k);

/*
 * gTop-k tournament over P sparse sets (P workers simulated on one GPU).
 *   in_idx     device, int32[P][k_in], each row strictly ascending, values in
 *              [0, n) (checked on the device: TOPK_EF_ERR_BAD_INPUT)
 *   in_val     device, fp32[P][k_in]
 *   P          number of workers, 1 <= P <= 512
 *   k_in       entries per input set, 0 <= k_in <= n
 *   k          entries kept per round and in the result, k >= 0
 *   n          index bound
 *   out_idx    device, int32[k]; the result in ascending index order; slots
 *              past the result length hold -1
 *   out_val    device, fp32[k]; the summed values; slots past the length 0
 *   out_count  device, int32[1]; the result length min(k, |S_0|)
 *   ws         device workspace of ws_bytes >=
 *              gtopk_merge_workspace_bytes(P, k_in, k)
 */
int gtopk_merge(const int32_t* in_idx, const float* in_val, int32_t P,
                int64_t k_in, int64_t k, int64_t n, int32_t* out_idx,
                float* out_val, int32_t* out_count, void* ws, size_t ws_bytes,
                void* stream);

/* ---------------------------------------------------------------- status */

/* ------------------------------------------- after the gTop-k merge */

/* Workspace bytes for gtopk_residual_return (a status block). */
size_t gtopk_residual_return_workspace_bytes(void);

/*
 * Residual return after gTop-k: only the global set updates the model ("A
 * Distributed Synchronous SGD Algorithm with Global Top-k Sparsification
 * for Low Bandwidth Networks", ABSTRACT), so each worker puts back into its
 * memory the values it sent whose index is not in the global set (error
 * feedback: what is not transmitted accumulates locally, "The Convergence of
 * Sparsified Gradient Methods", abstract):
 *     for every worker p and sent (i, v) with i not in global_idx:
 *         residual[p][i] = residual[p][i] + v          (one fp32 add)
 *   sent_idx    device, int32[P][k_sent], each row strictly ascending in [0, n)
 *               (the sets the workers sent, as given to gtopk_merge)
 *   sent_val    device, fp32[P][k_sent]
 *   global_idx  device, int32[k_global], strictly ascending in [0, n) (the
 *               first out_count indices gtopk_merge returned)
 *   residual    device, fp32[P][n], row p is worker p's memory
 *   ws          device workspace of >= gtopk_residual_return_workspace_bytes()
 * Malformed rows or global list: TOPK_EF_ERR_BAD_INPUT through
 * topk_ef_last_device_status(ws); no memory outside residual is written.
 * Errors: TOPK_EF_ERR_INVALID_ARG (P < 1, sizes out of range, null or
 * misaligned pointers), TOPK_EF_ERR_WORKSPACE, TOPK_EF_ERR_CUDA.
 */
int gtopk_residual_return(const int32_t* sent_idx, const float* sent_val,
                          int32_t P, int64_t k_sent, const int32_t* global_idx,
                          int64_t k_global, float* residual, int64_t n,
                          void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for topk_allgather_sum; 0 for invalid sizes
   (1 <= P <= 256, 0 <= k_in <= n <= 2^31 - 1). */
size_t topk_allgather_workspace_bytes(int32_t P, int64_t k_in, int64_t n);

/*
 * Top-k aggregation by AllGather, the O(kP) method the gTop-k review
 * measures its merge against ("A Distributed Synchronous SGD Algorithm with
 * Global Top-k Sparsification for Low Bandwidth Networks", ABSTRACT: current
 * methods use AllGather to accumulate the sparse gradients), on one GPU:
 * every worker's set is gathered and summed into a dense gradient in rank
 * order,
 *     out[i] = +0.0f;  for p = 0..P-1, for (i, v) in set p: out[i] += v
 * (one fp32 add each, in that order).
 *   in_idx   device, int32[P][k_in], rows strictly ascending in [0, n)
 *   in_val   device, fp32[P][k_in]
 *   out      device, fp32[n], written in full
 *   ws       device workspace of >= topk_allgather_workspace_bytes(P, k_in, n)
 * Malformed rows: TOPK_EF_ERR_BAD_INPUT through topk_ef_last_device_status;
 * no memory outside out is written.
 */
int topk_allgather_sum(const int32_t* in_idx, const float* in_val, int32_t P,
                       int64_t k_in, int64_t n, float* out, void* ws,
                       size_t ws_bytes, void* stream);

/* -------------------------------------------------------------- embedding */

/* Element types of the calls below (the calls above are fp32 throughout). */
#define TOPK_EF_F32 0
#define TOPK_EF_BF16 1
#define TOPK_EF_F16 2

/* Workspace bytes for embedding_lookup (a status block). */
size_t embedding_lookup_workspace_bytes(void);

/*
 * Embedding lookup with scaling, the forward pass of the layer whose gradient
 * is row-sparse:
 *     out[t][j] = round(scale * weight[ids[t]][j])     (fp32 product, one
 *                                                       rounding to out_type)
 *   weight     device, [V][ld_weight] of weight_type, the first D columns of
 *              each row are read; rows on 16-byte boundaries take the
 *              vectorised path (likewise out), others a path with identical
 *              results
 *   ids        device, int32[T] (id_bytes = 4) or int64[T] (id_bytes = 8)
 *   out        device, [T][ld_out] of out_type; columns from D on are not
 *              written; must not overlap weight
 *   sizes      0 <= T, V <= 2^31 - 1; 0 <= D <= 2^24; ld_weight, ld_out >= D
 *   ws         device workspace of >= embedding_lookup_workspace_bytes()
 * An id outside [0, V) gives a row of zeros and TOPK_EF_ERR_BAD_INPUT through
 * topk_ef_last_device_status(ws); no memory outside weight is read.
 * Errors: TOPK_EF_ERR_INVALID_ARG (sizes, types, null or misaligned pointers),
 * TOPK_EF_ERR_WORKSPACE, TOPK_EF_ERR_CUDA.
 */
int embedding_lookup(const void* weight, int32_t weight_type, int64_t ld_weight,
                     const void* ids, int32_t id_bytes, int64_t T, int64_t V,
                     int64_t D, float scale, void* out, int32_t out_type,
                     int64_t ld_out, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for embedding_grad and embedding_grad_rows; 0 for invalid
   sizes. */
size_t embedding_grad_workspace_bytes(int64_t T, int64_t V, int64_t D);

/*
 * Gradient of embedding_lookup with respect to weight, by sorted tokens:
 *     grad_weight[v][j] = (accumulate ? grad_weight[v][j] : 0)
 *                         + scale * sum over t with ids[t] = v of grad_out[t][j]
 * The sums are held in fp32 and rounded once to grad_weight_type.  Their
 * order depends on the sizes and ids alone (no floating-point atomics).
 * With fp32 output the call writes straight into the bucket that
 * topk_ef_compress and topk_ef_compress_batched read.
 *   grad_out     device, [T][ld_grad_out] of grad_out_type
 *   padding_idx  positions with this id contribute nothing (their row is zero,
 *                or with accumulate left as it was); any value outside [0, V),
 *                e.g. -1, for none
 *   grad_weight  device, [V][ld_grad_weight]; without accumulate every row is
 *                written, with it only the rows of ids that occur; columns
 *                from D on are not written; must not overlap grad_out
 *   ws           device workspace of >= embedding_grad_workspace_bytes(T, V, D)
 * An id outside [0, V), other than padding_idx, contributes nothing and gives
 * TOPK_EF_ERR_BAD_INPUT through topk_ef_last_device_status(ws).
 * Otherwise as embedding_lookup.
 */
int embedding_grad(const void* grad_out, int32_t grad_out_type,
                   int64_t ld_grad_out, const void* ids, int32_t id_bytes,
                   int64_t T, int64_t V, int64_t D, float scale,
                   int64_t padding_idx, void* grad_weight,
                   int32_t grad_weight_type, int64_t ld_grad_weight,
                   int32_t accumulate, void* ws, size_t ws_bytes, void* stream);

/*
 * The same gradient as a row-sparse set (the row form of the index-sorted
 * sets that the merge calls take):
 *   out_rows   device, int32[min(T, V)]: the distinct ids that occur, without
 *              padding_idx, ascending
 *   out_val    device, [min(T, V)][ld_out_val] of out_val_type: row j is the
 *              gradient of weight row out_rows[j]
 *   out_count  device, int32[1]: their number; slots of out_rows and rows of
 *              out_val from it on are not written
 */
int embedding_grad_rows(const void* grad_out, int32_t grad_out_type,
                        int64_t ld_grad_out, const void* ids, int32_t id_bytes,
                        int64_t T, int64_t V, int64_t D, float scale,
                        int64_t padding_idx, int32_t* out_rows, void* out_val,
                        int32_t out_val_type, int64_t ld_out_val,
                        int32_t* out_count, void* ws, size_t ws_bytes,
                        void* stream);

/* ------------------------------------------------------------------- muon */

/* Workspace bytes for muon_update; 0 for invalid arguments. */
size_t muon_workspace_bytes(int32_t B, int64_t rows, int64_t cols,
                            int32_t out_type);

/*
 * Momentum and orthogonalisation of the updates of B matrices by
 * Newton-Schulz products (the Muon optimiser's update), each on its own:
 *     momentum = fmaf(mu, momentum, grad)
 *     u        = nesterov ? fmaf(mu, momentum, grad) : momentum
 *                (without momentum: u = grad)
 *     X        = u / (||u||_F + eps)
 *     steps times, with (a, b, c) = coef[3 i .. 3 i + 2]:
 *         A = X X^T;   X = a X + (b A + c A A) X
 *     out      = round(scale * X)
 * (a tall matrix is treated as its transpose.)  Sums are fp32 or wider.  With
 * fp32 and fp16 output every product keeps 22 bits of its operands, and the
 * result is about as exact as one in plain fp32 (1e-6 to 1e-5 of its norm off)
 * before its one rounding to the output type, in rows and columns of 1e-6 of the
 * largest ones too (below that they lose bits: 1e-4 off at 1e-8).  With bf16 output and a short side above 128
 * the products' operands are rounded to 11 bits.  That leaves the result 1.7e-3
 * to 2.5e-3 of its norm off for dense matrices, up to 4e-3 for sparse ones and
 * ones with one large row and up to 7e-3 for equal entries (the rounding to bf16
 * alone: 1.65e-3, equal entries 0.4e-3 to 3e-3), and single rows of sparse ones
 * up to 1.5e-2 (rounding: 4e-3).  Ask for fp32 output and round it where that
 * is too much: three times the products' time.  fp32 output may be part of the
 * flat buffer that topk_ef_compress and topk_ef_compress_batched read.
 *   grad       device, [B][rows][cols] of grad_type; rows ld_grad apart,
 *              matrices stride_grad apart
 *   momentum   device, fp32[B][rows][cols] contiguous, updated in place; or
 *              NULL; must not overlap grad or out
 *   B          0 <= B <= 65535;  0 <= rows, cols <= 2^20
 *   eps        >= 0
 *   coef       host, float[3 * steps], read before the call returns.  On the
 *              singular values that can occur (at most 1 at the start) every
 *              |x (a + b x^2 + c x^4)| must stay within 4 and every
 *              |b x^2 + c x^4| within 16
 *   steps      1 <= steps <= 64
 *   out        device, [B][rows][cols] of out_type; rows ld_out apart,
 *              matrices stride_out apart; may start where grad does (B > 1:
 *              with the same type and strides only), must not overlap it
 *              otherwise
 *   ws         device workspace of >= muon_workspace_bytes(B, rows, cols,
 *              out_type)
 * Infinities, NaNs: as the formulas give them (a NaN anywhere makes the whole
 * of its matrix NaN); the other matrices are not touched by them.
 * Errors: TOPK_EF_ERR_INVALID_ARG (sizes, types, coefficients, null or
 * misaligned pointers), TOPK_EF_ERR_WORKSPACE, TOPK_EF_ERR_CUDA.
 */
int muon_update(const void* grad, int32_t grad_type, int64_t ld_grad,
                int64_t stride_grad, float* momentum, int32_t B, int64_t rows,
                int64_t cols, float mu, int32_t nesterov, float eps,
                const float* coef, int32_t steps, float scale, void* out,
                int32_t out_type, int64_t ld_out, int64_t stride_out, void* ws,
                size_t ws_bytes, void* stream);

/* ------------------------------------------------------------- layer norm */

/*
 * Layer norm of T rows:
 *     mean = 1/D sum x;  rstd = 1 / sqrt(1/D sum (x - mean)^2 + eps)
 *     out  = round((x - mean) rstd weight + bias)
 * Sums are fp32, the variance a sum of squared differences (an offset common to
 * a row costs no bits), one rounding to out_type.
 *   x          device, [T][ld_x] of x_type
 *   weight     device, [D] of weight_type, or NULL for 1
 *   bias       device, [D] of bias_type, or NULL for 0
 *   sizes      0 <= T <= 2^31 - 1; 1 <= D <= 2^24; ld_x, ld_out >= D
 *   eps        >= 0
 *   out        device, [T][ld_out] of out_type; columns from D on are not
 *              written; may be x itself (same type size and stride), must not
 *              overlap it otherwise
 *   mean, rstd device, fp32[T], or NULL: what layer_norm_grad needs
 * Rows on 16-byte boundaries with D a multiple of 8 take the vectorised path,
 * others an elementwise one (same formulas; sums in another order).
 * Infinities and NaNs make their row NaN, no other row.  There is no workspace.
 * Errors: TOPK_EF_ERR_INVALID_ARG (sizes, types, null or misaligned pointers, an
 * output that shares memory with another argument, but for what is said above),
 * TOPK_EF_ERR_CUDA.
 */
int layer_norm(const void* x, int32_t x_type, int64_t ld_x, const void* weight,
               int32_t weight_type, const void* bias, int32_t bias_type,
               int64_t T, int64_t D, float eps, void* out, int32_t out_type,
               int64_t ld_out, float* mean, float* rstd, void* stream);

/* Workspace bytes for layer_norm_grad (a status block, always OK after a call, and
   partial sums); 0 for invalid sizes. */
size_t layer_norm_grad_workspace_bytes(int64_t T, int64_t D);

/*
 * Gradient of layer_norm.  With xh = (x - mean) rstd and g = grad_out weight:
 *     grad_x      = round(rstd (g - 1/D sum g - xh 1/D sum (g xh)))
 *     grad_weight = (accumulate ? grad_weight : 0) + sum over rows of grad_out xh
 *     grad_bias   = (accumulate ? grad_bias : 0) + sum over rows of grad_out
 * Sums are fp32 in an order that depends on the sizes and alignment alone (no
 * floating-point atomics), rounded once.  fp32 weight gradients may be part of
 * the flat buffer that topk_ef_compress and topk_ef_compress_batched read.
 *   grad_out   device, [T][ld_grad_out] of grad_out_type
 *   x          device, [T][ld_x] of x_type: layer_norm's input
 *   mean, rstd device, fp32[T]: layer_norm's (far from 0 the rounding of mean leaves
 *              xh off by 2^-24 |mean| rstd, as x's own rounding does there)
 *   weight     as in layer_norm
 *   grad_x     device, [T][ld_grad_x] of x_type; may be x or grad_out itself
 *              (same type size and stride), must not overlap them otherwise
 *   grad_weight, grad_bias  device, [D] of their types; either or both may be
 *              NULL; written after all other arguments are read
 *   ws         device workspace of >= layer_norm_grad_workspace_bytes(T, D);
 *              not used (may be NULL) if grad_weight and grad_bias are NULL
 * Otherwise as layer_norm.
 */
int layer_norm_grad(const void* grad_out, int32_t grad_out_type,
                    int64_t ld_grad_out, const void* x, int32_t x_type,
                    int64_t ld_x, const float* mean, const float* rstd,
                    const void* weight, int32_t weight_type, int64_t T,
                    int64_t D, void* grad_x, int64_t ld_grad_x,
                    void* grad_weight, int32_t grad_weight_type,
                    void* grad_bias, int32_t grad_bias_type,
                    int32_t accumulate, void* ws, size_t ws_bytes,
                    void* stream);

/* ----------------------------------------------- losses over a vocabulary */

/* Workspace bytes for token_logprobs and token_logprobs_grad (a status block). */
size_t token_logprobs_workspace_bytes(void);

/*
 * Log-probabilities of given tokens, entropies and the largest alternatives of T
 * rows of logits.  With p = softmax(scale * logits[t]) (sums in fp32):
 *     lse[t]     = log sum_i exp(scale * logits[t][i])
 *     logprob[t] = scale * logits[t][ids[t]] - lse[t]
 *     entropy[t] = -sum_i p_i log p_i                  (0 log 0 = 0)
 *     top_ids[t][0 .. top - 1]  the ids of the largest logits, descending, the lower
 *                id first among equal ones (-0 equals +0; NaN above +Inf)
 *     top_logprobs[t][j]        their log-probabilities
 *   logits     device, [T][ld_logits] of logits_type; rows may start anywhere
 *   ids        device, int32[T] or int64[T] (id_bytes 4 or 8); or NULL (then logprob
 *              too): no row is padding
 *   scale      1e-30 .. 1e30 (1 / temperature)
 *   padding_idx  rows with this id are not read: their logprob, entropy and lse
 *              are 0, their top_ids -1 and top_logprobs -Inf.  Any value, e.g. -1
 *   top        0 .. 128.  With top > 0: V <= 2^20 (16-bit logits) or 2^19 (fp32), less
 *              64.  Slots past V get -1 and -Inf
 *   logprob, entropy, lse  device, fp32[T], each may be NULL
 *   top_ids, top_logprobs  device, int32 and fp32[T][top], each may be NULL
 *   sizes      0 <= T <= 2^31 - 1; 1 <= V <= 2^24; ld_logits >= V
 *   ws         device workspace of >= token_logprobs_workspace_bytes()
 * -Inf (a forbidden token) has probability 0, and one below 2^-126 of the largest
 * logit's counts as 0 in the sums.  A row of nothing else than -Inf has lse and
 * logprob -Inf and entropy 0.  NaN or +Inf makes a row's logprob, entropy, lse
 * and top_logprobs NaN, those of tokens at -Inf too; its top_ids follow the order
 * above.  An id outside [0, V), other than padding_idx, gives logprob 0 and
 * TOPK_EF_ERR_BAD_INPUT through topk_ef_last_device_status(ws); nothing outside
 * logits is read.
 * Errors: TOPK_EF_ERR_INVALID_ARG (sizes, types, null or misaligned pointers,
 * outputs or a workspace that share memory with another argument),
 * TOPK_EF_ERR_WORKSPACE, TOPK_EF_ERR_CUDA.
 */
int token_logprobs(const void* logits, int32_t logits_type, int64_t ld_logits,
                   const void* ids, int32_t id_bytes, int64_t T, int64_t V,
                   float scale, int64_t padding_idx, int32_t top,
                   float* logprob, float* entropy, float* lse,
                   int32_t* top_ids, float* top_logprobs, void* ws,
                   size_t ws_bytes, void* stream);

/*
 * Gradient of token_logprobs' log-probabilities and entropies in the logits:
 *     grad_logits[t][i] = scale * (grad_logprob[t] * ((i == ids[t]) - p_i)
 *                                  - grad_entropy[t] * p_i (log p_i + entropy[t]))
 * in fp32 (a p_i below 2^-126 counts as 0), one rounding to grad_logits_type.
 * p_i is exp(scale * logits[t][i] - lse[t]) while |lse[t]| <= 128, where lse's own
 * error leaves it off by 2^-16 at most.  Rows further from 0 (an offset, a small
 * temperature, nothing left but a mask of finite value) are summed again with exact
 * differences by one block each, which takes about 1.6 times as long where rows are
 * many, three times for one long row.
 *   lse        device, fp32[T], token_logprobs'
 *   entropy    device, fp32[T], token_logprobs'; needed with grad_entropy
 *   grad_logprob, grad_entropy  device, fp32[T]; NULL for 0
 *   grad_logits  device, [T][ld_grad_logits] of grad_logits_type; columns from V on are
 *              not written; may be logits itself (same type size and stride),
 *              must not overlap it otherwise.  Rows that lie in their
 *              128-byte lines as logits' do take the vectorised path
 * Rows that are padding or whose gradients are both 0 (an id outside [0, V) makes
 * grad_logprob 0) are not read and give zeros.  So do rows of nothing else than -Inf.
 * Otherwise as token_logprobs.
 */
int token_logprobs_grad(const void* logits, int32_t logits_type,
                        int64_t ld_logits, const void* ids, int32_t id_bytes,
                        int64_t T, int64_t V, float scale, int64_t padding_idx,
                        const float* lse, const float* entropy,
                        const float* grad_logprob, const float* grad_entropy,
                        void* grad_logits, int32_t grad_logits_type,
                        int64_t ld_grad_logits, void* ws, size_t ws_bytes,
                        void* stream);

/* Workspace bytes for distill_loss (a status block). */
size_t distill_loss_workspace_bytes(void);

/*
 * Distillation from a teacher's top logits: a (ids, logits) set for each row, as
 * token_logprobs' top_ids and top_logprobs give it.  With
 * q = softmax(scale * teacher_logits[t]) over its K entries and
 * p = softmax(scale * logits[t]) over all V tokens (sums in fp32):
 *     loss[t]           = weight[t] * sum_k q_k (log q_k - log p_{teacher_ids[t][k]})
 *     grad_logits[t][i] = weight[t] * scale * (p_i - sum of q_k with id i)
 * (the gradient of the sum of loss: a temperature's square and a mean's divisor
 * belong into weight).
 *   teacher_ids     device, int32 or int64 [T][K]; a negative id is an empty entry; an
 *                   id may occur more than once
 *   teacher_logits  device, [T][K] of teacher_type; -Inf has q = 0
 *   K               0 .. 256
 *   weight          device, fp32[T], or NULL for 1
 *   loss            device, fp32[T], or NULL; may be weight itself
 *   grad_logits     device, [T][ld_grad_logits] of grad_logits_type, or NULL; as in
 *                   token_logprobs_grad
 *   ws              device workspace of >= distill_loss_workspace_bytes()
 * Rows whose weight is 0 or that have no entry above -Inf give loss 0 and zeros;
 * those of weight 0 are not read.  The loss with and without grad_logits may differ in
 * its last bits (sums in another order).  An id >= V is an empty entry and gives
 * TOPK_EF_ERR_BAD_INPUT through topk_ef_last_device_status(ws).
 * Infinite and NaN logits, sizes, scale and errors as in token_logprobs; a teacher's
 * token at -Inf makes the loss +Inf.
 */
int distill_loss(const void* logits, int32_t logits_type, int64_t ld_logits,
                 const void* teacher_ids, int32_t id_bytes,
                 const void* teacher_logits, int32_t teacher_type, int64_t T,
                 int64_t V, int32_t K, float scale, const float* weight,
                 float* loss, void* grad_logits, int32_t grad_logits_type,
                 int64_t ld_grad_logits, void* ws, size_t ws_bytes,
                 void* stream);

/* Synchronises `stream` and returns the device-side status of the last call
   that used `ws`: TOPK_EF_OK, TOPK_EF_ERR_DEVICE_TIMEOUT,
   TOPK_EF_ERR_BAD_INPUT or TOPK_EF_ERR_INTERNAL (or TOPK_EF_ERR_CUDA if the
   read-back failed). */
int topk_ef_last_device_status(const void* ws, void* stream);

/* The cudaError_t of the last TOPK_EF_ERR_CUDA returned on this thread. */
int topk_ef_last_cuda_error(void);

/* Human-readable name of a return code (static string). */
const char* topk_ef_status_string(int status);

/*
 * Diagnostics of the last compress call on `ws` (synchronises `stream`):
 *   info[0]  path taken: 0 = candidate prefilter, 1 = full rescan fallback
 *            (a small tensor: 1 = the previous call's threshold did not
 *            decide the top k, so every block ran the exact select)
 *   info[1]  candidates kept by the prefilter
 *   info[2]  candidate capacity of the workspace
 *   info[3]  kernels launched by that call
 *   info[4]  1 if the k-th key's relative digit-1 bin of some tensor held
 *            more candidates than its entry list, so the select kernel took
 *            the exact-count exchange (one more grid barrier); else 0
 *   info[5]  reserved (0)
 * `info` is host memory of 6 int64.  Returns a status code.
 */
int topk_ef_path_info(const void* ws, void* stream, int64_t* info);

/*
 * Diagnostics of the last compress call on `ws` (synchronises `stream`), in
 * nanoseconds; -1 for a step that did not run.  `ns` is host memory of 20
 * int64.  ns[0..7]: block 0 of the select kernel, from the kernel's start:
 *   candidate path: ns[4] offset look-back done, ns[5] gather done,
 *     ns[1] first grid barrier, ns[2] second grid barrier, ns[3] barrier of
 *     the exact-count exchange (only when a bin overflowed its entry list),
 *     ns[6] emission starts, ns[7] end;
 *   rescan fallback: ns[1] gather barrier, ns[3..5] the barriers after
 *     digit passes 1..3, ns[6] the count barrier, ns[7] end.
 * ns[8..10]: the sampling block of the first tensor, from its start: samples
 * loaded, first histogram level resolved, end.
 * ns[11..14], over all blocks and from the moment the first block of the
 * streaming pass got past its wait on the setup kernel: the last streaming
 * block done, the first select (or threshold) block started, block 0 of that
 * kernel started, its last block done; then, latest over the blocks of that
 * kernel: block started, output offset known (candidate path), candidates
 * gathered, arrived at the barrier after the entry lists.  ns[19] is
 * reserved (-1).
 */
int topk_ef_phase_times(const void* ws, void* stream, int64_t* ns);

/*
 * Test hook, process wide: bit 0 forces the full rescan fallback of the
 * compress calls; bit 1 forces the prefilter threshold of every tensor to 0
 * (every element a candidate, which overflows the candidate capacity for
 * large tensors and so also ends in the fallback); bit 2 makes the grid-wide
 * exchange of a single-tensor compress call wait for one block more than
 * the grid has, so that its bounded wait runs out (after about a second) and
 * the call records TOPK_EF_ERR_DEVICE_TIMEOUT, with undefined outputs, and
 * makes the products of muon_update wait for an event that never comes (two
 * seconds a launch, the same status); bits 3..5, when 1, 2, 3 or 4, make the
 * rounds of gtopk_merge that one thread-block cluster per pair can hold use
 * clusters of 16, 14, 12 or 8 CTAs wherever that size can run (else the size
 * is chosen per round as usual).  0 restores normal behaviour.  Returns the previous flags.  The flags are
 * process-wide state read by every call in the process (the library's only
 * state outside the caller's workspace besides the tracing record and the
 * scratch array of topk_ef_compress_static): set them only in tests, with no
 * other calls in flight.
 */
int topk_ef_set_test_flags(int flags);

/*
 * Tracing, process wide, for one thread at a time: while enabled, every
 * kernel a compute call launches is bracketed by two CUDA events recorded on
 * the call's stream (the library owns the events, created on the device that
 * is current when tracing is enabled).  Up to 4096 launches are recorded;
 * later ones are not.
 *   topk_ef_trace_enable(1|0)   switch on / off (either clears the record)
 *   topk_ef_trace_read(ms, names, max, &count)
 *       waits for the recorded launches, writes the duration in milliseconds
 *       (host float[max]) and kernel name (host const char*[max], static
 *       strings) of the first min(max, recorded) of them, sets *count to that
 *       number and clears the record.
 *   topk_ef_trace_only(name, every)    record only the launches of the
 *       kernel with this name (as topk_ef_trace_read reports it, e.g.
 *       "stream_kernel"), and of those the 1st, (every+1)-th, ... after
 *       tracing was enabled, so that the other launches keep running back to
 *       back; NULL or "" selects every kernel again.  The string is copied.
 *       every < 1: TOPK_EF_ERR_INVALID_ARG.
 */
int topk_ef_trace_enable(int on);
int topk_ef_trace_read(float* ms, const char** names, int max_entries, int* count);
int topk_ef_trace_only(const char* kernel_name, int every);

#ifdef __cplusplus
}
#endif

#endif /* TOPK_EF_H */

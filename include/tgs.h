/*
 * tgs.h -- C ABI of the MI355X (gfx950) error-feedback top-k gradient
 * sparsifier.
 *
 * The operations come from these web pages (cited by title and section):
 *   [EF]    arxivdaily listing for arXiv 2004.05298, entry "Sparsified SGD with
 *           Memory": top-k compression with the accumulated error kept in
 *           memory and added back before the next compression.
 *   [CONV]  same listing, entry "The Convergence of Sparsified Gradient
 *           Methods": sort by magnitude, send a subset, accumulate the rest
 *           locally.
 *   [SORT]  same listing, entry "Empirical Analysis on Top-k Gradient
 *           Sparsification for Distributed Deep Learning in a Supercomputing
 *           Environment": gradient sorting on the GPU is what makes top-k slow.
 *   [HT]    same listing, entry "Rethinking gradient sparsification as total
 *           error minimization": hard-threshold sparsifier (k set by a constant
 *           threshold) with error feedback.
 *   [LAYER] fugumt page for arXiv 2502.07634, related-paper entry "L-GreCo:
 *           Layerwise-Adaptive Gradient Compression for Efficient and
 *           Accurate Deep Learning": compression applied layer by layer, each
 *           layer with its own degree.
 *   [GTOPK] nubint review "A Distributed Synchronous SGD Algorithm with Global
 *           Top-k Sparsification for Low Bandwidth Networks", ABSTRACT and
 *           Method: global top-k of the largest |values| over P workers by an
 *           O(log P)-round tournament; only the selected indices survive.
 *   [EST]   arxivdaily listing, entry "Near-Optimal Sparse Allreduce for
 *           Distributed Deep Learning" (top-k picked through an estimated
 *           threshold rather than a sort); fugumt page for arXiv 2502.07634,
 *           related-paper entry "An Efficient Statistical-based Gradient
 *           Compression Technique for Distributed Training Systems"
 *           (threshold sparsification with an estimated threshold) and its
 *           Abstract (top-k's sorting costs offset what it saves).
 *   [RTOPK] arxivdaily listing, entry "rTop-k: A Statistical Estimation
 *           Approach to Distributed SGD": random-k chained after top-k.
 *
 * Conventions shared by every entry point
 *   - Array arguments are DEVICE pointers owned by the caller; the library
 *     keeps no pointer after the call returns and allocates no device memory.
 *   - Calls are asynchronous on `stream` (0 = the null stream); nothing waits
 *     for the device except tgs_check_device_error().
 *   - Only 4-byte alignment is required.  Inputs whose grad/residual
 *     pointers differ in alignment modulo 16 bytes take a slower scalar path.
 *   - n is at most 2^31 - 1, so every index fits in int32.  Indices are
 *     relative to the pointers passed.
 *   - `workspace` is caller-owned device memory of at least the size the
 *     matching *_workspace_bytes() query returns.  One workspace serves one
 *     call at a time; calls that share a workspace must be ordered (same
 *     stream).  Its first 32 KB (the header) hold the device error word and
 *     the synchronisation state of the top-k kernels; the rest is scratch.
 *     A workspace is ready after tgs_workspace_init() (a kernel, so it may
 *     sit in a captured graph) or after being zero-filled, and every call
 *     leaves it ready for the next one, on the host's order or replayed
 *     from a graph: the library keeps no state on the host.  Between calls
 *     the caller must not write to the header.  Any of the operations may
 *     use a workspace after any other.
 *   - Device error word (the header's first word): kernels only set bits in
 *     it, so it collects every problem since it was last read;
 *     tgs_check_device_error() reads and clears it.  After a report other
 *     than bad merge input, run tgs_workspace_init() before the next call.
 *   - Residency: the top-k kernels that synchronise their workgroups through
 *     memory (k_step, k_rank, k_general) size their grid to what fits on the device
 *     at once and assume every workgroup runs concurrently.  Kernels running
 *     on other streams at the same time can keep workgroups from starting;
 *     the waits are bounded, so the call then ends with wrong outputs and the
 *     wait-timeout bit (0x2) in the device error word, never a hang.  Run
 *     the top-k step while no other kernel occupies the device, or check
 *     the error word.
 *   - Magnitude order: key(x) = bits(x) & 0x7FFFFFFF as an unsigned integer.
 *     This matches |x| for every non-NaN value, ranks NaN above infinity and
 *     makes -0 and +0 equal.  Among equal keys the lower index comes first.
 *   - acc = residual + grad is one binary32 add, rounded to nearest even,
 *     never fused and never flushed to zero.
 *   - On a negative status nothing has been enqueued and the outputs are
 *     untouched; tgs_last_error() describes the reason.
 */
#ifndef TGS_H
#define TGS_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t tgs_status;
#define TGS_OK 0
#define TGS_EINVAL (-1)     /* bad size, null pointer, overlapping buffers, bad lambda */
#define TGS_EWORKSPACE (-2) /* workspace smaller than the query returned             */
#define TGS_EHIP (-3)       /* a HIP launch failed; see tgs_last_error()              */
#define TGS_EDEVICE (-4)    /* a kernel flagged a wait timeout or inconsistent counts */

/* Bytes of workspace tgs_topk_ef_step needs for this (n, k).  0 if the sizes
   are invalid. */
size_t tgs_topk_workspace_bytes(int64_t n, int64_t k);

/*
 * Error-feedback top-k step ([EF], [CONV]; the selection replaces the full
 * sort that [SORT] identifies as the bottleneck).  For k up to ~48k and
 * n >= 2^19 it is one kernel launch that reads grad and residual once;
 * n <= 2^18 with k <= 256 is one launch too; other sizes take an exact
 * radix-select path (three launches).  Every route gives the same result.
 *   grad      [n] float32, read only.
 *   residual  [n] float32, in/out: on entry the accumulated error, on exit
 *             acc with the selected entries set to +0.0f.
 *   k         0 <= k <= n entries are selected: the first k of all n indices
 *             ordered by (key(acc) descending, index ascending).
 *   out_idx   [k] int32, out: the selected indices in that order.
 *   out_val   [k] float32, out: acc at out_idx, bit for bit.
 * grad must not overlap residual or the outputs; the outputs must not overlap
 * each other or residual.  k == 0 only writes residual = acc.
 */
tgs_status tgs_topk_ef_step(const float* grad, float* residual, int64_t n, int64_t k,
                            int32_t* out_idx, float* out_val, void* workspace,
                            size_t workspace_bytes, hipStream_t stream);

/*
 * tgs_topk_ef_step for callers that cannot allocate device memory (code under
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same step, with no workspace argument.  Its workspace is a device array of
 * TGS_NOALLOC_WORKSPACE_BYTES inside the library, one per GPU, held until the
 * process ends; sizes whose tgs_topk_workspace_bytes(n, k) exceed it are
 * rejected with TGS_EINVAL.  The call allocates nothing: on a device's first
 * call it looks up that device's copy of the array and zero-fills its header
 * with a kernel on `stream`.  All calls on one GPU share the array (it keeps
 * the last call's contents), so calls that overlap in time on one GPU race:
 * order them on one stream.  Its device error word is not reachable; callers
 * that need it use tgs_topk_ef_step.
 */
#define TGS_NOALLOC_WORKSPACE_BYTES ((size_t)64 << 20)
tgs_status tgs_topk_ef_step_noalloc(const float* grad, float* residual, int64_t n, int64_t k, int32_t* out_idx,
                                    float* out_val, hipStream_t stream);

/* Bytes of workspace tgs_topk_ef_step_segmented needs for this segment table
   (HOST arrays, as below).  0 if the table is invalid. */
size_t tgs_topk_segmented_workspace_bytes(int32_t nseg, const int64_t* offsets, const int64_t* ks);

/*
 * Layer-wise error-feedback top-k ([LAYER] with [EF], [CONV]): the vector
 * grad/residual [offsets[nseg]] is cut into nseg segments (layers) and each
 * gets the top-k step of tgs_topk_ef_step with its own k, in one call.
 *   offsets   HOST int64 [nseg + 1]: segment s is [offsets[s], offsets[s+1]);
 *             offsets[0] == 0, nondecreasing, offsets[nseg] <= 2^31 - 1.
 *   ks        HOST int64 [nseg]: 0 <= ks[s] <= the segment's length.
 *   out_idx / out_val  [sum of ks]: segment s's pairs start at
 *             sum(ks[0..s)), in the order tgs_topk_ef_step gives them, with
 *             indices relative to the segment's start.
 * Segments of at most 2^18 entries with k <= 256 run together, up to 64 per
 * launch of one kernel; every other segment takes its own step.  The
 * results are those of one tgs_topk_ef_step call per segment.  Pointer and
 * overlap rules as tgs_topk_ef_step, over the whole vector and sum(ks).
 */
tgs_status tgs_topk_ef_step_segmented(const float* grad, float* residual, int32_t nseg,
                                      const int64_t* offsets, const int64_t* ks, int32_t* out_idx,
                                      float* out_val, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream);

/* Bytes of workspace tgs_threshold_ef_step needs for this n (0 if invalid). */
size_t tgs_threshold_workspace_bytes(int64_t n);

/*
 * Hard-threshold step with error feedback ([HT]).
 *   An entry qualifies when key(acc_i) >= key((float)lambda); lambda must be a
 *   non-negative, non-NaN number.
 *   out_idx/out_val [capacity]: the first min(count, capacity) qualifying
 *             entries (i, acc_i) in ascending index order.
 *   d_count   device int64, out: the total number of qualifying entries
 *             (which may exceed capacity).
 *   residual  in/out: +0.0f at every emitted index, acc everywhere else
 *             (qualifying entries beyond the capacity keep acc).
 */
tgs_status tgs_threshold_ef_step(const float* grad, float* residual, int64_t n, float lambda,
                                 int32_t* out_idx, float* out_val, int64_t capacity,
                                 int64_t* d_count, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* Bytes of workspace tgs_threshold_estimate needs for m samples (0 if m is
   outside [1, 2^24]).  A workspace of the larger of this and
   tgs_threshold_workspace_bytes(n) serves both calls of an estimated step. */
size_t tgs_threshold_estimate_workspace_bytes(int64_t m);

/*
 * Threshold estimate from a sample ([EST]), for the hard-threshold step.
 *   sample_idx [m] int32, device: positions in [0, n) (repeats allowed), for
 *             example drawn uniformly by the caller; 1 <= m <= 2^24.
 *   q         1 <= q <= m: the estimate is the q-th largest of
 *             key(residual[s_j] + grad[s_j]) over j < m (ties counted), so a
 *             target density rho takes q = ceil(rho * m).
 *   d_lambda  device float, out: the float whose bits are that key (>= 0).
 * grad and residual are only read.  A position outside [0, n) sets the
 * bad-input bit of the device error word (the estimate is then unspecified).
 * Two launches.  The workspace must be 256-byte aligned.
 */
tgs_status tgs_threshold_estimate(const float* grad, const float* residual, int64_t n, const int32_t* sample_idx,
                                  int64_t m, int64_t q, float* d_lambda, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream);

/*
 * tgs_threshold_ef_step with the threshold read on the device ([HT] fed by
 * [EST]): an entry qualifies when key(acc_i) >= key(*d_lambda), read when the
 * kernels run (so tgs_threshold_estimate may write it earlier on the same
 * stream, with no host round trip).  Any bit pattern is accepted: the key of
 * a negative value is that of its magnitude; a NaN's key is only reached by
 * NaNs of at least its payload.  Everything else as tgs_threshold_ef_step.
 */
tgs_status tgs_threshold_ef_step_dev(const float* grad, float* residual, int64_t n, const float* d_lambda,
                                     int32_t* out_idx, float* out_val, int64_t capacity, int64_t* d_count,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace tgs_rtopk_ef_step needs (0 if the sizes are invalid). */
size_t tgs_rtopk_workspace_bytes(int64_t n, int64_t r, int64_t k);

/*
 * rTop-k step with error feedback ([RTOPK] with [EF]): k entries drawn
 * uniformly at random from the r of largest |acc|.
 *   0 <= k <= r <= n.  The top r are the first r by (key(acc) desc, index
 *   asc), as tgs_topk_ef_step finds them.  Entry i draws u_i = output word 0
 *   of Philox4x32-10 (Salmon et al., SC'11) at counter (i, step & 0xFFFFFFFF,
 *   step >> 32, 0) under key (seed & 0xFFFFFFFF, seed >> 32); the k of the top
 *   r with the smallest (u_i, i) are sent.
 *   out_idx/out_val [k]: the sent entries in (key desc, index asc) order,
 *             values bit for bit.
 *   residual  in/out: +0.0f at the k sent, acc everywhere else (the r - k
 *             passed over included).
 * r = k gives tgs_topk_ef_step's result.  Two more kernels follow the top-r
 * step's launches.  Pointer and overlap rules as tgs_topk_ef_step.
 */
tgs_status tgs_rtopk_ef_step(const float* grad, float* residual, int64_t n, int64_t r, int64_t k, uint64_t seed,
                             uint64_t step, int32_t* out_idx, float* out_val, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* Bytes of workspace tgs_gtopk_merge needs (0 if the sizes are invalid). */
size_t tgs_gtopk_workspace_bytes(int32_t P, int64_t k, int64_t n);

/*
 * gTop-k tournament of P workers' sparse sets on one GPU ([GTOPK]).
 *   idx [P][k] int32, val [P][k] float32: worker p's k pairs, any order;
 *             indices must be distinct within a row and inside [0, n).
 *   Round r = 0, 1, ... while 2^r < P: slot s (s a multiple of 2^(r+1))
 *   absorbs slot s + 2^r when that slot exists: the union by index, values of
 *   a shared index added in binary32, keeps its first k entries by (key desc,
 *   index asc).  A slot without a partner passes through.
 *   out_idx/out_val [k]: slot 0 after the last round, in (key desc, index
 *             asc) order.
 *   out_mask [P][k] uint8: 1 where idx[p][j] is one of out_idx, else 0.
 * Rows that break the index precondition set a device error word; check it
 * with tgs_check_device_error (the outputs are then unspecified).
 * k is at most 2^20 and P k at most 2^31 - 1; the workspace must be 16-byte
 * aligned.  Each call starts by zero-filling the part of the workspace it
 * keeps its tables and counters in, so it assumes nothing of that part.
 */
tgs_status tgs_gtopk_merge(const int32_t* idx, const float* val, int32_t P, int64_t k, int64_t n,
                           int32_t* out_idx, float* out_val, uint8_t* out_mask, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* -------------------------------------------------------------------------
 * Operators of the training step around the sparsifier: the token embedding
 * (whose dense gradient the top-k step compresses) and the Muon update of the
 * weight matrices.  They hold values in the types below, compute in fp32 and
 * round once, to nearest even, where they store.  The conventions above hold,
 * except that arrays need only their own type's alignment and workspaces must
 * be 256-byte aligned.
 * ------------------------------------------------------------------------- */
typedef int32_t tgs_dtype;
#define TGS_FP32 0
#define TGS_BF16 1
#define TGS_FP16 2
#define TGS_INT32 3
#define TGS_INT64 4

/* Bytes of workspace tgs_embedding_lookup needs (0 if T is invalid). */
size_t tgs_embedding_lookup_workspace_bytes(int64_t T);

/*
 * Embedding lookup with scaling: out[t][:] = scale * table[tokens[t]][:].
 *   tokens    [T] int32 or int64.  A negative token is a masked place: its
 *             row is +0.  A token >= V sets the bad-input bit of the device
 *             error word, and its row is +0.
 *   table     [V][D] fp32, bf16 or fp16, row-major.
 *   out       [T][D] fp32, bf16 or fp16: fp32(table) * scale, rounded once.
 * 0 <= T, 1 <= V, 1 <= D, each at most 2^31 - 1; scale is finite.  Sizes that
 * would take a launch of 2^32 threads (2^34 16-byte vectors of out) are refused.
 */
tgs_status tgs_embedding_lookup(const void* tokens, tgs_dtype tokens_dtype, int64_t T, const void* table,
                                tgs_dtype table_dtype, int64_t V, int64_t D, float scale, void* out,
                                tgs_dtype out_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace tgs_embedding_grad needs (0 if the sizes or types are
   invalid): 16 bytes a place for the sort, and two partial rows for every 8
   to 64 places; the header alone for few places of a small table. */
size_t tgs_embedding_grad_workspace_bytes(int64_t T, int64_t V, int64_t D, tgs_dtype grad_dtype, tgs_dtype out_dtype);

/*
 * Gradient of the lookup with respect to the table, by sorted tokens:
 *   S[v][:] = scale * sum of grad[t][:] over the places with tokens[t] == v
 *   accumulate == 0: out = S, rows that no token names are +0
 *   accumulate != 0: out = out + S, rows that no token names are not touched
 * The sums are fp32, in an order that depends on the tokens alone, so equal
 * inputs give equal bits.  Masked places (negative tokens) and tokens >= V
 * (bad-input bit) add to nothing: their rows of grad may hold anything.  Sizes
 * that would take a launch of 2^32 threads are refused, as the lookup's are.
 */
tgs_status tgs_embedding_grad(const void* tokens, tgs_dtype tokens_dtype, int64_t T, const void* grad,
                              tgs_dtype grad_dtype, int64_t V, int64_t D, float scale, void* out, tgs_dtype out_dtype,
                              int32_t accumulate, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace tgs_newton_schulz needs (0 if the sizes or the type are
   invalid): 10 bytes an entry of x (padded to 128 a side, 4 of them to the
   update's tiles of up to 256) and 4 of the smaller square with bf16, 16 and 8
   with fp32 and fp16, and up to 8 MB for sums that workgroups share. */
size_t tgs_newton_schulz_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, tgs_dtype dtype);

/*
 * Orthogonalises a stack of matrices by Newton-Schulz products: for each
 *   X <- x / (|x|_F + eps), then `steps` times
 *   A = X X^T,  X <- a X + (b A + c A^2) X        (X^T X where rows > cols)
 *   x, out    [batch][rows][cols] of one type (fp32, bf16, fp16).  out may be
 *             x itself, and must not overlap it otherwise.
 * 1 <= batch <= 65535, 1 <= rows, cols <= 65536, 1 <= steps <= 64, eps >= 0.
 * Coefficients with which a singular value that starts in [0, 1] could pass
 * 2^30 are refused.  The products use fp16 operands scaled by powers of two
 * and fp32 sums.  fp32 and fp16 results, and bf16 ones whose shorter side is at
 * most 32, are as exact as with fp32 products (three fp16 products each).  Other
 * bf16 results take single products: before the final rounding (1.7e-3 of the
 * 2-norm) they are off by at most half of that for matrices like gradients, whose
 * singular values fall off into noise.  Matrices of low rank come out up to 1.6e-3
 * off where the shorter side is 33 to 64, 5e-3 at 65, 3e-3 at 128, 2e-3 at 256 and
 * 1.4e-3 at 512.  A NaN or infinity in x makes its matrix's result NaN.  Equal
 * inputs give equal bits.
 */
tgs_status tgs_newton_schulz(const void* x, tgs_dtype dtype, int64_t batch, int64_t rows, int64_t cols, int32_t steps,
                             float a, float b, float c, float eps, void* out, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* Bytes of workspace tgs_muon_step needs (0 if the sizes or the type are
   invalid): what tgs_newton_schulz needs for the weights' type. */
size_t tgs_muon_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, tgs_dtype weight_dtype);

/*
 * One Muon step for a stack of weight matrices:
 *   momentum <- beta momentum + grad
 *   u = grad + beta momentum (nesterov != 0), or momentum
 *   O = u orthogonalised as tgs_newton_schulz does
 *   weight <- (1 - lr weight_decay) weight - lr sqrt(max(1, rows / cols)) O
 *   weight    [batch][rows][cols] fp32, bf16 or fp16, in/out; rows are taken
 *             to be a layer's outputs.
 *   grad      [batch][rows][cols] fp32, bf16 or fp16, read only.
 *   momentum  [batch][rows][cols] fp32, in/out.
 * The arrays must not overlap.  Sizes, coefficients, exactness (by the
 * weights' type) as tgs_newton_schulz.
 */
tgs_status tgs_muon_step(void* weight, tgs_dtype weight_dtype, const void* grad, tgs_dtype grad_dtype, float* momentum,
                         int64_t batch, int64_t rows, int64_t cols, float lr, float beta, int32_t nesterov,
                         float weight_decay, int32_t steps, float a, float b, float c, float eps, void* workspace,
                         size_t workspace_bytes, hipStream_t stream);

/* -------------------------------------------------------------------------
 * Operators over rows, between a model's hidden states and its losses.  The
 * conventions of the section above hold.
 * ------------------------------------------------------------------------- */

/*
 * Layer norm of each row: out = (x - mean) rstd weight + bias with mean = sum x
 * / D and rstd = 1 / sqrt(sum (x - mean)^2 / D + eps).
 *   x         [T][D] fp32, bf16 or fp16; out [T][D] of any of them, x itself
 *             included where the types agree.
 *   weight, bias  [D] of one type, fp32, bf16 or fp16; either may be null (1, 0).
 *   mean, rstd    [T] float, out, for the gradients; either may be null.
 * 0 <= T <= 2^31 - 1, 1 <= D <= 2^24, eps >= 0.  The mean is known before the
 * squares are summed, and where the values lie flat around it (within a 256th of
 * it) the roundings of its sum are taken off: a large mean costs no more than x's
 * own rounding, and a row of one value gives the bias.  Rows whose sum or squares
 * pass fp32's range, or fall below it beside as small an eps, are normed too.  A
 * row's NaN or infinity makes the whole row NaN.
 */
tgs_status tgs_layer_norm(const void* x, tgs_dtype x_dtype, int64_t T, int64_t D, const void* weight, const void* bias,
                          tgs_dtype weight_dtype, float eps, void* out, tgs_dtype out_dtype, float* mean, float* rstd,
                          hipStream_t stream);

/* Bytes of workspace tgs_layer_norm_grad needs (0 if the sizes are invalid): up
   to 1,280 partial rows of 2 D floats, 34 MB or one row (8 D bytes: 134 MB for
   2^24 columns) at most. */
size_t tgs_layer_norm_grad_workspace_bytes(int64_t T, int64_t D);

/*
 * Gradients of the layer norm, with xh = (x - mean) rstd and gw = grad weight:
 *   grad_x      = rstd (gw - sum gw / D - xh sum (gw xh) / D)
 *   grad_weight = sum over rows of grad xh,  grad_bias = sum over rows of grad
 *   grad      [T][D] fp32, bf16 or fp16; x, mean, rstd, weight as given to and
 *             left by tgs_layer_norm.
 *   grad_x    [T][D] of x's type; x itself, or grad where the types agree, included.
 *   grad_weight, grad_bias  [D] of param_dtype; either may be null.
 * The sums over rows are fp32, in an order that depends on the sizes and types
 * alone: equal inputs give equal bits.  x - mean need be no fp32 number.
 */
tgs_status tgs_layer_norm_grad(const void* grad, tgs_dtype grad_dtype, const void* x, tgs_dtype x_dtype, int64_t T,
                               int64_t D, const float* mean, const float* rstd, const void* weight,
                               tgs_dtype weight_dtype, void* grad_x, void* grad_weight, void* grad_bias,
                               tgs_dtype param_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace tgs_token_logprobs needs (0 if the sizes or the type are
   invalid): the header, and what slices of rows leave where rows are few. */
size_t tgs_token_logprobs_workspace_bytes(int64_t T, int64_t V, tgs_dtype dtype, int32_t top);

/*
 * Log probabilities of given tokens under p = softmax(logits / temperature).
 *   logits    [T] rows of V scores, fp32, bf16 or fp16, `ld` elements from row to
 *             row (ld >= V; what lies between rows is not read).
 *   tokens    [T] int32 or int64.  A negative token is a masked place: its row
 *             is not needed, and its results are +0 and -1.  A token >= V sets
 *             the bad-input bit of the device error word and is masked too.
 *   logprobs  [T] float: log p(token).
 *   stats     [T][2] float: (r, l) with log sum e^(logits / temperature) = r /
 *             temperature + l, for the gradient; here r is the largest score.
 *   entropy   [T] float: -sum p log p; may be null.
 *   top_indices, top_logprobs  [T][top] int32 and float: the `top` largest
 *             scores of each row, ties to the lower index, and their log
 *             probabilities; 0 <= top <= min(64, V).
 * 1e-6 <= temperature <= 1e6.  A score of -inf has no probability (its log is
 * -inf and it adds nothing to the entropy); the type's lowest finite value is a
 * score like any other.  A row of which every score is -inf has log
 * probabilities of -inf and entropy 0.  NaN or +inf in a row makes its
 * log probabilities and entropy NaN; among alternatives a NaN ranks above all.
 * Equal calls give equal bits.
 */
tgs_status tgs_token_logprobs(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                              const void* tokens, tgs_dtype tokens_dtype, float temperature, float* logprobs,
                              float* stats, float* entropy, int32_t top, int32_t* top_indices, float* top_logprobs,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The gradient of the logits:
 *   out = (grad_logprobs (onehot(token) - p) - grad_entropy p (log p + entropy)) / temperature
 *   stats     as tgs_token_logprobs left them; entropy too where grad_entropy is given.
 *   grad_logprobs, grad_entropy  [T] float; either may be null, not both.
 *   out       [T] rows of V of the logits' type, ld_out elements apart (what lies
 *             between rows is left as it is); the logits themselves with ld_out
 *             == ld included.
 * Rows of masked places, and rows of which every score is -inf, are +0.  NaN or
 * +inf in a row of any other place makes its gradient NaN.  The workspace is a
 * header (32 KB).
 */
tgs_status tgs_token_logprobs_grad(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                   const void* tokens, tgs_dtype tokens_dtype, float temperature, const float* stats,
                                   const float* grad_logprobs, const float* entropy, const float* grad_entropy,
                                   void* out, int64_t ld_out, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/* Bytes of workspace tgs_distillation_loss and tgs_distillation_loss_and_grad
   need (0 if the sizes or the type are invalid). */
size_t tgs_distillation_workspace_bytes(int64_t T, int64_t V, tgs_dtype dtype);

/*
 * Distillation from a teacher's top logits: KL(q || p) of each row with p =
 * softmax(logits / temperature) over all V and q = softmax(teacher /
 * temperature) over the row's slots,
 *   loss = sum over slots of q (log q - log p(index)).
 *   logits, ld  as tgs_token_logprobs.
 *   indices   [T][K] int32 or int64: the tokens of the teacher's K slots, 1 <=
 *             K <= 1024, in any order; a negative one is an empty slot, one >= V
 *             sets the bad-input bit and is empty too.  An index may stand in
 *             several slots.
 *   teacher   [T][K] fp32, bf16 or fp16 scores (logits, or log probabilities:
 *             what they have in common cancels); -inf gives a slot q = 0.
 *   loss      [T] float.  +inf where a slot with q > 0 has a student's score of -inf.
 *   stats     [T][2] float as tgs_token_logprobs', for the gradient; may be null.
 * A row without a slot of q > 0 is a masked place: loss 0, gradient +0, its
 * logits not needed.  NaN in a row's logits, or in its teacher's scores, and
 * +inf in either make its loss and gradient NaN.
 */
tgs_status tgs_distillation_loss(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                 const void* indices, tgs_dtype indices_dtype, const void* teacher,
                                 tgs_dtype teacher_dtype, int64_t K, float temperature, float* loss, float* stats,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The gradient of the logits: out = grad_loss (p - q) / temperature, where q
 * sums the slots that name a token.
 *   grad_loss [T] float; stats as tgs_distillation_loss left them.
 *   out, ld_out  as tgs_token_logprobs_grad, the logits themselves included.
 * Rows of which every score is -inf are +0; those of NaN, alone or among -inf, are
 * NaN, from this call and from the one below.  The workspace is a header (32 KB).
 */
tgs_status tgs_distillation_grad(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                 const void* indices, tgs_dtype indices_dtype, const void* teacher,
                                 tgs_dtype teacher_dtype, int64_t K, float temperature, const float* stats,
                                 const float* grad_loss, void* out, int64_t ld_out, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);

/*
 * Both in one call, for rows whose weights are known: the losses, and in out the
 * gradient of sum over rows of weights loss (weights [T] float, or null for 1).
 * A row's second reading follows its first, so that LDS and the caches serve what
 * they still hold of it; the two calls above read all rows from memory twice.
 */
tgs_status tgs_distillation_loss_and_grad(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                          const void* indices, tgs_dtype indices_dtype, const void* teacher,
                                          tgs_dtype teacher_dtype, int64_t K, float temperature, const float* weights,
                                          float* loss, void* out, int64_t ld_out, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream);

/* Waits for `stream`, then reads and clears the device error word of
   `workspace`: TGS_OK if no kernel flagged a problem since it was last read,
   TGS_EINVAL for an input index outside its range (a merge row's index out
   of range or repeated, a sample position out of range), TGS_EDEVICE for a
   wait that timed out or inconsistent counts.  Works for every workspace.
   Synchronous: not for use inside graph capture. */
tgs_status tgs_check_device_error(const void* workspace, hipStream_t stream);

/* Makes `workspace` ready for any operation: zero-fills its header (the first
   min(workspace_bytes, 32 KB) bytes) with a kernel on `stream`.  Needed once
   for memory that is not zero-filled (and after a TGS_EDEVICE report); the
   calls themselves keep the workspace ready. */
tgs_status tgs_workspace_init(void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Static text for a status code. */
const char* tgs_status_string(tgs_status s);

/* Thread-local description of the last failure on the calling thread ("" if
   none). */
const char* tgs_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* TGS_H */

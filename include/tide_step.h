/*
 * tide_step.h -- C ABI of the training-step operators next to the collectives, on MI355X (gfx950).
 *
 * The reduce-scatter (tide.h) reads per-parameter bf16 gradients in place and leaves flat fp32
 * shards.  This library holds the operators on either side of it that work on the same tensors:
 *
 *   - layer norm and embedding lookup with their gradients: the parameter gradients that are sums
 *     over tokens, written once, as bf16 or fp32, where the reduce-scatter reads them;
 *   - the global L2 norm over many tensors and clipping by it: what a step does to the shards
 *     before the optimizer;
 *   - what tokens pass through in the blocks between, with gradients: the experts of a mixture (tokens
 *     sorted by expert and back, with weights), rotary positions of several axes, dropout.
 *
 * Conventions for every entry point (as in tide.h):
 *   - Device pointers are HIP device addresses on the current device; host arrays are read only
 *     during the call and may be freed as soon as it returns.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).  Calls are
 *     stream-ordered and asynchronous and only launch kernels: no allocation, copy, event or
 *     synchronisation, so every call may be captured into a HIP graph and replayed on the buffers'
 *     contents of the moment.  No state is kept between calls.
 *   - `workspace` is caller-owned device memory of at least the bytes that the query of the same
 *     name gives, 16-byte aligned; its contents need no initialisation and mean nothing after the
 *     call.  Calls that may run at the same time need workspaces of their own.
 *   - Inputs are never written; outputs must not overlap inputs or each other unless stated.  Blocks of
 *     columns of one buffer, of one row stride, do not overlap; matrices of different row strides count
 *     as overlapping where their first and last elements do.
 *   - Results do not depend on scheduling: sums have a fixed order for given sizes, and no
 *     floating-point atomic is used.
 *   - Errors are returned as tide_status, before any work is enqueued except TIDE_ERR_HIP; nothing
 *     is printed and nothing is thrown.  tide_step_last_hip_error() gives the HIP error code behind
 *     the calling thread's most recent TIDE_ERR_HIP.
 *   - Tensors start on element boundaries; 16-byte-aligned ones are read and written fastest.
 */
#ifndef TIDE_STEP_H
#define TIDE_STEP_H

#include <stdint.h>

#include "tide.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum {
  TIDE_BF16 = 0,
  TIDE_FP32 = 1,
  TIDE_INT32 = 2, /* token and expert ids, positions */
  TIDE_INT64 = 3  /* token and expert ids, positions */
};

/*
 * Global norm of a list of gradient tensors.
 *   num_tensors  >= 0
 *   grads        host [num_tensors]: contiguous device tensors (NULL allowed only for empty ones);
 *                tensors may overlap (each then counts)
 *   numels       host [num_tensors], elements of each, >= 0
 *   dtype        TIDE_BF16 or TIDE_FP32
 *   sumsq        device, one double, 8-byte aligned, or NULL
 *   norm         device, one float, 4-byte aligned, or NULL
 * Result: sumsq = sum of squares of every element, norm = sqrt(sumsq) rounded to fp32; 0 for no
 * elements.  Squares and sums are held in 64 bits, so no finite gradient overflows; a NaN or an
 * infinity anywhere gives NaN or infinity.  A data-parallel job adds up `sumsq` over its ranks and
 * passes the total to tide_grad_clip.
 * Errors: TIDE_ERR_INVALID (null or misaligned pointer, negative count, unknown dtype, total above
 * 2^42 elements, workspace too small or misaligned, sumsq, norm or workspace over a gradient or each
 * other), TIDE_ERR_HIP.
 */
int64_t tide_grad_norm_workspace(int32_t num_tensors, const int64_t* numels, int32_t dtype); /* bytes; -1: bad argument */
tide_status tide_grad_norm(int32_t num_tensors, const void* const* grads, const int64_t* numels, int32_t dtype,
                           double* sumsq, float* norm, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Clipping by a given sum of squares.
 *   sumsq     device, one double: the sum of squares over all ranks' gradients
 *   max_norm  >= 0, may be infinity, not NaN
 *   outs      host [num_tensors]: where tensor i goes, contiguous, of the gradients' type; outs[i] may
 *             be grads[i] (in place) and must otherwise not overlap any gradient or output
 *   norm      device, one float, or NULL; not within a gradient, output or *sumsq
 * Result: with n = sqrt(sumsq) and c = min(1, max_norm / (n + 1e-6)) in 64 bits, rounded to fp32,
 * outs[i][k] = grads[i][k] * c, one fp32 product rounded to the tensors' type; norm = n.  A NaN or
 * infinite n gives c = NaN or 0 (NaN where max_norm is infinite too), as the formula says.
 * Errors: as tide_grad_norm; TIDE_ERR_INVALID also for overlaps and a max_norm below 0 or NaN,
 * TIDE_ERR_NOMEM where the host has no memory for the check of overlaps.
 */
tide_status tide_grad_clip(int32_t num_tensors, const void* const* grads, void* const* outs, const int64_t* numels,
                           int32_t dtype, const double* sumsq, double max_norm, float* norm, void* stream);

/* Norm and clipping in one call, for gradients that are all on this device: tide_grad_norm's sum,
 * then tide_grad_clip by it.  `sumsq` and `norm` may be NULL; workspace as tide_grad_norm. */
tide_status tide_clip_grad_norm(int32_t num_tensors, const void* const* grads, void* const* outs,
                                const int64_t* numels, int32_t dtype, double max_norm, double* sumsq, float* norm,
                                void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Layer norm over the last dimension.
 *   rows, cols    rows >= 0, 1 <= cols < 2^31
 *   x, x_stride   device, row i starts at element i * x_stride (>= cols)
 *   dtype         of x and y: TIDE_BF16 or TIDE_FP32
 *   weight, bias  device [cols], contiguous, of param_dtype; either may be NULL (1 and 0)
 *   eps           finite, >= 0
 *   y, y_stride   device, as x
 *   mean, rstd    device [rows] fp32, or NULL
 * Result: mean = sum(x) / cols, var = sum((x - mean)^2) / cols, rstd = 1 / sqrt(var + eps),
 * y = (x - mean) * rstd * weight + bias, all in fp32, y rounded once.
 * Errors: TIDE_ERR_INVALID (null or misaligned pointer, sizes, strides, unknown dtype, eps, y
 * overlapping x or a parameter), TIDE_ERR_HIP.
 */
tide_status tide_layer_norm(int64_t rows, int64_t cols, const void* x, int64_t x_stride, int32_t dtype,
                            const void* weight, const void* bias, int32_t param_dtype, float eps, void* y,
                            int64_t y_stride, float* mean, float* rstd, void* stream);

/*
 * Gradient of tide_layer_norm.
 *   dy, x         device, `dtype`, with row strides as above
 *   weight        device [cols] of param_dtype, or NULL (1)
 *   mean, rstd    device [rows] fp32, as tide_layer_norm wrote them
 *   dx, dx_stride device, `dtype`, or NULL (not wanted); may be dy itself with the same stride (in place)
 *   dweight, dbias device [cols] of param_dtype, contiguous, or NULL (not wanted)
 * Result, with xhat = (x - mean) * rstd and g = dy * weight, in fp32:
 *   dx = rstd * (g - sum(g) / cols - xhat * sum(g * xhat) / cols), rounded once;
 *   dweight = sum over rows of dy * xhat, dbias = sum over rows of dy (0 for no rows), rounded once.
 * Errors: as tide_layer_norm; TIDE_ERR_INVALID also for a workspace too small or misaligned.
 */
int64_t tide_layer_norm_bwd_workspace(int64_t rows, int64_t cols, int32_t dtype); /* bytes; -1: bad argument */
tide_status tide_layer_norm_bwd(int64_t rows, int64_t cols, const void* dy, int64_t dy_stride, const void* x,
                                int64_t x_stride, int32_t dtype, const void* weight, int32_t param_dtype,
                                const float* mean, const float* rstd, void* dx, int64_t dx_stride, void* dweight,
                                void* dbias, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Embedding lookup with scaling.
 *   tokens        0 <= tokens < 2^31
 *   ids           device [tokens], contiguous, of ids_dtype (TIDE_INT32 or TIDE_INT64)
 *   vocab, dim    table rows (0 <= vocab < 2^31) and columns (1 <= dim < 2^31)
 *   table         device [vocab, dim], contiguous, of dtype (TIDE_BF16 or TIDE_FP32)
 *   scale         fp32
 *   out           device [tokens, dim], contiguous, of dtype
 * Result: out[t] = table[ids[t]] * scale in fp32, rounded once; +0 where ids[t] is outside
 * [0, vocab) -- a padded position, or a token of another rank's rows -- without reading the table.
 * Errors: TIDE_ERR_INVALID (null or misaligned pointer, sizes, unknown dtype, overlap), TIDE_ERR_HIP.
 */
tide_status tide_embedding(int64_t tokens, const void* ids, int32_t ids_dtype, int64_t vocab, int64_t dim,
                           const void* table, int32_t dtype, float scale, void* out, void* stream);

/*
 * Gradient of tide_embedding with respect to the table, every row of it.
 *   dy            device [tokens, dim], contiguous, of dtype
 *   dtable        device [vocab, dim], contiguous, of dtype
 *   accumulate    0: dtable is written, zero rows included; 1: the gradient is added to it (a table
 *                 that is also the output projection, gradients summed over micro-batches)
 * Result: dtable[v] = scale * (sum of dy[t] over the t with ids[t] = v) [+ the old dtable[v]], in
 * fp32, rounded once.  The tokens of a row are taken in ascending t and summed in parts, the parts' sums
 * in an order that is fixed for given ids and sizes.  With accumulate, rows of no token are
 * neither read nor written.  Ids outside [0, vocab) contribute nothing.
 * Errors: as tide_embedding; TIDE_ERR_INVALID also for a workspace too small or misaligned.
 */
int64_t tide_embedding_bwd_workspace(int64_t tokens, int64_t vocab, int64_t dim); /* bytes; -1: bad argument */
tide_status tide_embedding_bwd(int64_t tokens, const void* ids, int32_t ids_dtype, int64_t vocab, int64_t dim,
                               const void* dy, int32_t dtype, float scale, int32_t accumulate, void* dtable,
                               void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Experts of a mixture.  Each of `tokens` tokens has `choices` experts; a (token, choice) pair is numbered
 * token * choices + choice.  tide_expert_sort brings the pairs into the order of their experts and gives
 * each a row of a sorted buffer:
 *
 *   offsets[e]   where the rows of expert e start: offsets[0] = 0, offsets[e + 1] = offsets[e] + the number
 *                of its pairs, rounded up to a multiple of `align`
 *   place[p]     the row of pair p, or -1 where its id is outside [0, experts): a padded token, or an
 *                expert of another rank
 *   source[r]    the pair of row r, or -1 for a row of no pair: behind an expert's pairs up to its
 *                multiple, and behind the last expert
 *
 * The pairs of an expert keep their order.  A token may name an expert twice.
 *   tokens, choices   tokens >= 0, 1 <= choices <= TIDE_MAX_CHOICES, fewer than 2^31 pairs
 *   experts, align    1 <= experts <= TIDE_MAX_EXPERTS, align >= 1
 *   ids               device [tokens, choices], contiguous, of ids_dtype (TIDE_INT32 or TIDE_INT64)
 *   place             device [tokens, choices]
 *   source, rows      device [rows]; rows is at least tide_expert_rows(), which any ids fit, and below 2^31
 *   offsets           device [experts + 1]
 * Errors: TIDE_ERR_INVALID (null or misaligned pointer, sizes, too few rows, unknown dtype, workspace,
 * overlap), TIDE_ERR_HIP.
 */
#define TIDE_MAX_CHOICES 64
#define TIDE_MAX_EXPERTS 2048
int64_t tide_expert_rows(int64_t tokens, int32_t choices, int32_t experts, int32_t align); /* -1: bad argument */
int64_t tide_expert_sort_workspace(int64_t tokens, int32_t choices, int32_t experts);      /* bytes; -1: bad argument */
tide_status tide_expert_sort(int64_t tokens, int32_t choices, const void* ids, int32_t ids_dtype, int32_t experts,
                             int32_t align, int32_t* place, int32_t* source, int64_t rows, int32_t* offsets,
                             void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Tokens into the sorted buffer: out[r] = x[source[r] / choices], zeros for a row of no pair.
 *   x, x_stride       device [tokens, dim], row i starts at element i * x_stride (>= dim)
 *   dtype             of x and out: TIDE_BF16 or TIDE_FP32
 *   place, source     as tide_expert_sort wrote them; no address outside the tensors is read or written
 *                     for any others
 *   out, out_stride   device [rows, dim], as x
 * Its gradient is tide_expert_combine without weights.
 * Errors: TIDE_ERR_INVALID (null or misaligned pointer, sizes, strides, unknown dtype, overlap), TIDE_ERR_HIP.
 */
tide_status tide_expert_dispatch(int64_t tokens, int32_t choices, int64_t dim, const void* x, int64_t x_stride,
                                 int32_t dtype, const int32_t* place, const int32_t* source, int64_t rows, void* out,
                                 int64_t out_stride, void* stream);

/*
 * The sorted buffer's rows back at their tokens: y[t] = sum over j of weights[t, j] * x[place[t, j]], in
 * fp32 in ascending j, rounded once.  Pairs without a row count as nothing (their weights are not used),
 * and a token of none is zeros.  Rows of no pair are not read.
 *   x, x_stride       device [rows, dim] of dtype
 *   weights           device [tokens, choices], contiguous, of weight_dtype (TIDE_BF16 or TIDE_FP32); NULL: ones
 *   y, y_stride       device [tokens, dim] of dtype
 */
tide_status tide_expert_combine(int64_t tokens, int32_t choices, int64_t dim, const void* x, int64_t x_stride,
                                int64_t rows, int32_t dtype, const void* weights, int32_t weight_dtype,
                                const int32_t* place, void* y, int64_t y_stride, void* stream);

/*
 * Gradients of tide_expert_combine.
 *   dx[r] = weights[source[r]] * dy[source[r] / choices] in fp32, rounded once; zeros for a row of no pair
 *   dweights[t, j] = sum over the columns of dy[t] * x[place[t, j]] in fp32, rounded once; 0 without a row
 *   dy                device [tokens, dim] of dtype
 *   dx                device [rows, dim] of dtype; may be x itself with the same stride (in place)
 *   dweights          device [tokens, choices], contiguous, of weight_dtype
 */
tide_status tide_expert_combine_bwd(int64_t tokens, int32_t choices, int64_t dim, const void* dy, int64_t dy_stride,
                                    const void* x, int64_t x_stride, int64_t rows, int32_t dtype, const void* weights,
                                    int32_t weight_dtype, const int32_t* place, const int32_t* source, void* dx,
                                    int64_t dx_stride, void* dweights, void* stream);

/*
 * Rotary positions of several axes (text: one; image: height, width; video: time, height, width).
 *   tokens, heads, dim  0 <= tokens < 2^31, 0 <= heads <= TIDE_ROTARY_MAX_HEADS, 1 <= dim <= TIDE_ROTARY_MAX_DIM
 *   x                 device, element (t, h, c) at t * x_token_stride + h * x_head_stride + c; strides >= 0
 *   dtype             of x and out: TIDE_BF16 or TIDE_FP32
 *   positions         device [axes, tokens], contiguous, of positions_dtype (TIDE_INT32, TIDE_INT64 or TIDE_FP32)
 *   axes, sections    1 <= axes <= TIDE_ROTARY_MAX_AXES; host [axes]: how many pairs turn with each axis,
 *                     >= 1, P of them in all with 2 P <= dim; pairs are numbered through, axis after axis
 *   freqs             device [P] fp64, 8-byte aligned: the angle of a pair for one step along its axis
 *   pairing           TIDE_ROTARY_HALVES: pair i is elements i and P + i of a head;
 *                     TIDE_ROTARY_NEIGHBOURS: elements 2 i and 2 i + 1
 *   inverse           0, or 1 to turn back: the gradient with respect to x
 *   out               device, as x with strides of its own, its elements apart from each other; may be x
 *                     itself with the same strides (in place)
 * Result: with a = positions[axis of i][t] * freqs[i], both as fp64 and their product (minus that for inverse),
 * and cos a, sin a rounded to fp32, off by less than 2^-35 before that, pair (u, v) becomes
 * (u cos a - v sin a, v cos a + u sin a) in fp32, rounded once.  That holds for |a| up to 2^64; beyond, a sine and
 * cosine of some angle are taken.  Elements from 2 P on are copied.  A position that is infinite or NaN gives NaN.
 * Errors: TIDE_ERR_INVALID (null or misaligned pointer, sizes, strides, unknown dtype, pairing or
 * inverse, overlap), TIDE_ERR_HIP.
 */
#define TIDE_ROTARY_MAX_HEADS 65535
#define TIDE_ROTARY_MAX_DIM 1024
#define TIDE_ROTARY_MAX_AXES 8
enum { TIDE_ROTARY_HALVES = 0, TIDE_ROTARY_NEIGHBOURS = 1 };
tide_status tide_rotary(int64_t tokens, int64_t heads, int64_t dim, const void* x, int64_t x_token_stride,
                        int64_t x_head_stride, int32_t dtype, const void* positions, int32_t positions_dtype,
                        int32_t axes, const int32_t* sections, const double* freqs, int32_t pairing, int32_t inverse,
                        void* out, int64_t out_token_stride, int64_t out_head_stride, void* stream);

/*
 * Dropout by a counter-based generator, added to a residual; the mask is stored nowhere and made again by
 * the same seed and offset.
 *   rows, cols        rows >= 0, 1 <= cols < 2^44; element (i, k) is number e = offset + i * cols + k
 *   x, x_stride       device, row i starts at element i * x_stride (>= cols)
 *   dtype             of x, residual and out: TIDE_BF16 or TIDE_FP32
 *   p                 in [0, 1]; t = p * 65536 rounded to the nearest whole number (ties to even)
 *   seed              64 bits; seed_device (device, one int64, 8-byte aligned), where not NULL, holds it
 *                     instead, so that a captured call can be replayed with another
 *   offset            >= 0, offset + rows * cols <= 2^62: a rank's part of a larger tensor, a call's part of a
 *                     step's numbers
 *   residual          device, as x, or NULL (zeros)
 *   out, out_stride   device, as x; may be x or the residual itself with the same stride (in place)
 * Philox4x32 with 10 rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011), key = the
 * seed's low and high 32 bits, counter = (low, high 32 bits of e / 8, 0, 0), gives four words; u = 16 bits
 * of them, word (e mod 8) / 2, its low half for an even e.
 * Result: x * (65536 / (65536 - t)) + residual where u >= t, else the residual; in fp32, rounded once.  An
 * element that is dropped counts as zero whatever it holds.  The probability is t / 65536 exactly, and the
 * scale is that probability's.  The gradient is the same call on dy without a residual.
 * Errors: TIDE_ERR_INVALID (null or misaligned pointer, sizes, strides, unknown dtype, p, offset, overlap),
 * TIDE_ERR_HIP.
 */
tide_status tide_dropout(int64_t rows, int64_t cols, const void* x, int64_t x_stride, int32_t dtype, double p,
                         uint64_t seed, const int64_t* seed_device, int64_t offset, const void* residual,
                         int64_t residual_stride, void* out, int64_t out_stride, void* stream);

/* HIP error code (hipError_t value) behind the calling thread's last TIDE_ERR_HIP of this library, 0 if none. */
int32_t tide_step_last_hip_error(void);

/* Build id of this library (see tide_build_id). */
const char* tide_step_build_id(void);

#ifdef __cplusplus
}
#endif

#endif /* TIDE_STEP_H */

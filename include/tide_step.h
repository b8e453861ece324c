/*
 * tide_step.h -- C ABI of the training-step operators next to the collectives, on MI355X (gfx950).
 *
 * The reduce-scatter (tide.h) reads per-parameter bf16 gradients in place and leaves flat fp32
 * shards.  This library holds the operators on either side of it that work on the same tensors:
 *
 *   - layer norm and embedding lookup with their gradients: the parameter gradients that are sums
 *     over tokens, written once, as bf16 or fp32, where the reduce-scatter reads them;
 *   - the global L2 norm over many tensors and clipping by it: what a step does to the shards
 *     before the optimizer.
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
  TIDE_INT32 = 2, /* token ids */
  TIDE_INT64 = 3  /* token ids */
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

/* HIP error code (hipError_t value) behind the calling thread's last TIDE_ERR_HIP of this library, 0 if none. */
int32_t tide_step_last_hip_error(void);

/* Build id of this library (see tide_build_id). */
const char* tide_step_build_id(void);

#ifdef __cplusplus
}
#endif

#endif /* TIDE_STEP_H */

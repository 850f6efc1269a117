/*
 * ringsim_ops.h -- C ABI of libringsim's training- and serving-step operators:
 * what a rank computes on either side of its collectives, on device tensors
 * of one MI355X (gfx950).
 *
 *   - ringsim_rms_norm: root-mean-square norm of every row, with the
 *     residual's addition in front of it and, on request, an output in 8 bits
 *     with scales (what follows an all-reduce of partial products);
 *   - ringsim_rms_norm_backward: its gradients;
 *   - ringsim_grad_norm, ringsim_scale_grads, ringsim_clip_grads: the 2-norm of
 *     all gradients together and the clipping by it (what follows the
 *     all-reduce or reduce-scatter of the gradient buckets).
 *
 * Conventions shared by every call:
 *   - Result codes, streams and their meaning are those of ringsim.h: a call
 *     checks its arguments on the host, enqueues kernels on `stream` and
 *     returns; nothing waits for the device. An argument that is refused is
 *     refused before anything is enqueued (RINGSIM_INVALID_ARGUMENT).
 *   - Structures and host arrays are read during the call only. Device memory
 *     is the caller's, must stay valid until the enqueued work is done, and
 *     must be on the current device.
 *   - No call allocates, and a call enqueues kernel launches only, so calls may
 *     be captured into a HIP graph; the captured graph holds the addresses of
 *     the call. Calls that share a workspace or write the same memory have to
 *     be ordered on the device.
 *   - Pointers need the alignment of their element type, no more; rows and
 *     tensors that start on a 16-byte boundary are faster.
 *   - Results do not depend on timing: the same call on the same values gives
 *     the same bits (no floating-point atomics).
 *   - Arithmetic is in fp32 (sums of squares of gradients in fp64), each
 *     result rounded once to its output's type, round to nearest even. Infinities and
 *     NaN take the course the formulas give them.
 */
#ifndef RINGSIM_OPS_H
#define RINGSIM_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "ringsim.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types that only these operators take, beside RINGSIM_FLOAT32 and
 * RINGSIM_BFLOAT16 of ringsim_datatype_t. FLOAT8_E4M3 is the OCP format
 * (largest value 448, no infinities), an output type only. */
typedef enum {
  RINGSIM_FLOAT16 = 16,
  RINGSIM_FLOAT8_E4M3 = 17
} ringsim_op_datatype_t;

/* Longest row the norm and its gradients take. */
#define RINGSIM_NORM_MAX_COLS 32768

/* Arguments of ringsim_rms_norm. Every tensor of rows is a [outer, inner, cols]
 * array whose last dimension is contiguous; its strides, in elements, are
 * given as {outer, inner} (inner strides are not read where inner == 1).
 * Rows of an output must not overlap. */
typedef struct {
  const void* x;           /* dtype */
  const void* residual;    /* dtype; NULL: none */
  const void* weight;      /* cols elements of weight_dtype; NULL: all ones */
  void* out;               /* out_dtype */
  void* residual_out;      /* dtype; x + residual, required with `residual`, else NULL */
  float* scales;           /* out_dtype FLOAT8_E4M3: [outer * inner, groups], contiguous; else NULL */
  int64_t x_stride[2];
  int64_t residual_stride[2];
  int64_t out_stride[2];
  int64_t residual_out_stride[2];
  int64_t outer;
  int64_t inner;
  int64_t cols;            /* 1 .. RINGSIM_NORM_MAX_COLS */
  int dtype;               /* FLOAT32, BFLOAT16 or FLOAT16 */
  int weight_dtype;        /* dtype or FLOAT32 */
  int out_dtype;           /* dtype or FLOAT8_E4M3 */
  int group;               /* columns a scale covers: 32, 64 or 128, or 0 = the whole row */
  float eps;               /* finite, >= 0 */
} ringsim_rms_norm_t;

/* Root-mean-square norm with the residual's addition. For every row:
 *     h = x + residual                       (or x)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 * residual_out receives h and out receives y, both computed from the sum
 * before it is rounded. With out_dtype FLOAT8_E4M3, out and scales receive,
 * for every group of `group` columns (the last one may be shorter; groups =
 * ceil(cols / group), or 1):
 *     scale = max(max|y| / 448, 2^-126),  q = y * (1 / scale)
 * so that q * scale stands for y; a NaN in a group makes its scale NaN. The
 * reciprocal and the product are fp32 values: q is y / scale rounded to
 * nearest, but where y / scale lies within 2^-22 of itself from the middle of
 * two 8-bit values it may be either of them.
 * residual_out, and out in the rows' type, may be x or residual themselves
 * (same address, same strides); otherwise outputs must not overlap inputs or
 * each other. A row whose sum of squares is beyond fp32's range gives zeros,
 * as 1 / sqrt(inf) does. Nothing to do (no rows) is a success. */
ringsim_result_t ringsim_rms_norm(const ringsim_rms_norm_t* args, ringsim_stream_t stream);

/* Arguments of ringsim_rms_norm_backward; tensors as in ringsim_rms_norm_t. */
typedef struct {
  const void* grad_out;      /* gradient of y, dtype */
  const void* h;             /* what the forward call normed: its residual_out, or x without a residual */
  const void* weight;        /* NULL: all ones */
  const void* grad_residual; /* gradient that reaches h past the norm, dtype; NULL: none */
  void* grad_in;             /* gradient of h (of x and of residual alike), dtype */
  void* grad_weight;         /* cols elements of weight_dtype; NULL: not wanted */
  void* workspace;           /* with grad_weight: ringsim_rms_norm_backward_workspace bytes, 16-byte aligned */
  size_t workspace_bytes;
  int64_t grad_out_stride[2];
  int64_t h_stride[2];
  int64_t grad_residual_stride[2];
  int64_t grad_in_stride[2];
  int64_t outer;
  int64_t inner;
  int64_t cols;
  int dtype;
  int weight_dtype;
  float eps;
} ringsim_rms_norm_backward_t;

/* Gradients of the norm. With r = 1 / sqrt(mean(h^2) + eps), recomputed from
 * h, n = h * r and g = grad_out * weight, for every row
 *     grad_in = grad_residual + r * (g - n * mean(g * n))
 * and over all rows
 *     grad_weight = sum of grad_out * n
 * where mean(g * n) is formed as r * mean(g * h): a row's sums of h^2 and of
 * g * h have to lie in fp32's range. Beyond it, r is 0 as in the forward call.
 * grad_weight is overwritten (with zeros if there are no rows). grad_in may
 * be grad_out, h or grad_residual itself (same address, same strides). The
 * gradient of an output in 8 bits passes its rounding unchanged: grad_out is
 * then the gradient of q * scale. */
ringsim_result_t ringsim_rms_norm_backward(const ringsim_rms_norm_backward_t* args, ringsim_stream_t stream);

/* Bytes of workspace ringsim_rms_norm_backward needs for `rows` = outer *
 * inner rows of `cols` elements of `dtype` when it writes grad_weight (0 for
 * few rows). Host only. */
ringsim_result_t ringsim_rms_norm_backward_workspace(int64_t rows, int64_t cols, int dtype, size_t* bytes);

/* The 2-norm of `ntensors` gradients together,
 *     *norm = |scale| * sqrt(sum over all elements of grad^2)
 * as one fp32 value in device memory. grads[i] holds counts[i] elements of
 * dtypes[i] (FLOAT32, BFLOAT16 or FLOAT16, which may differ from tensor to
 * tensor), contiguous; grads[i] may be NULL where counts[i] is 0. `scale`
 * (finite) is what the gradients are to be multiplied with: 1 / nranks after
 * a summing collective, 1 / the loss scale. Squares are summed in fp64, so
 * that neither large nor small values are lost; the result of no elements is
 * 0. A sharded gradient's norm takes the shards of all ranks in one call.
 * workspace: ringsim_grad_norm_workspace bytes of device memory, 16-byte
 * aligned. */
ringsim_result_t ringsim_grad_norm(int ntensors, const void* const* grads, const int64_t* counts, const int* dtypes,
                                   float scale, float* norm, void* workspace, size_t workspace_bytes,
                                   ringsim_stream_t stream);

/* Bytes of workspace ringsim_grad_norm and ringsim_clip_grads need for a list
 * (0 for short ones). Host only. */
ringsim_result_t ringsim_grad_norm_workspace(int ntensors, const int64_t* counts, const int* dtypes, size_t* bytes);

/* Scales gradients by what a norm known to the device leaves of them,
 *     outs[i] = grads[i] * scale * min(1, max_norm / (*norm + eps))
 * where a NaN norm makes every element NaN and an infinite one makes finite
 * elements 0. outs[i] is grads[i] itself or does not overlap any gradient, and
 * no two outputs overlap (a gradient that two parameters share is listed
 * once); outs == NULL means in place, where a factor of exactly 1 writes
 * nothing.
 * max_norm and eps are finite and >= 0. For ranks that hold copies of the
 * same gradients: the norm of one copy serves them all. */
ringsim_result_t ringsim_scale_grads(int ntensors, const void* const* grads, void* const* outs, const int64_t* counts,
                                     const int* dtypes, float scale, const float* norm, float max_norm, float eps,
                                     ringsim_stream_t stream);

/* ringsim_grad_norm and then ringsim_scale_grads with that norm, which is
 * also written to *norm, in one call. */
ringsim_result_t ringsim_clip_grads(int ntensors, const void* const* grads, void* const* outs, const int64_t* counts,
                                    const int* dtypes, float scale, float max_norm, float eps, float* norm,
                                    void* workspace, size_t workspace_bytes, ringsim_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RINGSIM_OPS_H */

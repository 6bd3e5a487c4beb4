/*
 * fs_layers.h -- C ABI of the layers around the matching on AMD MI355X (gfx950):
 * the layer norm of states with the residual sum in front of it, scores of
 * states held in 8-bit integers, and two losses on rows of scores (a teacher's
 * top logits, and a balanced use of the columns), each with its gradients.
 * Part of libfs_sinkhorn.so; status codes, stream and error conventions are
 * those of fs_sinkhorn.h.
 *
 * States that are matched are formed by layers; rows of scores are what the
 * solver's half-step normalises.  A converged plan's largest entries of each row
 * are a teacher for cheaper scores (distillation); where the solver holds the
 * columns' mass to a marginal, the balance loss asks for an even use of them.
 *
 * Conventions (every entry point of this file):
 *  - Tensors are device memory on the calling thread's current device.  Rows are
 *    given as fs_rows (fs_attention.h) of one head: a [batch][rows][width] view
 *    whose last axis is contiguous and whose other strides (in elements) are
 *    free; stride_head is not looked at.  Views whose rows are 16-byte aligned
 *    with a width of whole 16-byte chunks are read with wide loads (the layer
 *    norm's also where they start at whole dwords), others element by element.
 *    Arrays given by plain pointers are contiguous.  Outputs may not overlap
 *    themselves, one another, an input or the workspace (slices of one buffer side
 *    by side, of equal strides, do not; against an input whole extents count).
 *  - Work is enqueued on `stream` and is asynchronous; nothing synchronises,
 *    nothing is allocated, and every call may be captured into a graph (a replay
 *    uses the same buffers: two captured calls that may overlap need a workspace
 *    each).  Equal calls give equal bits: no sum depends on the order in which
 *    workgroups run.
 *  - Sums and statistics are fp32 (over workgroups' parts of a sum in 64 bits),
 *    sums of products of 8-bit integers exact; an output is rounded once.
 */
#ifndef FS_LAYERS_H
#define FS_LAYERS_H

#include "fs_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- layer norm ----------------------------------------------------------
 *   z = x + residual (rounded to dtype: the sum that goes on), or x
 *   mean = mean(z), rstd = 1 / sqrt(mean((z - mean)^2) + eps)
 *   y = weight (z - mean) rstd + bias
 * Rows i >= lengths[b] are padding: nothing depends on what they hold (a first few
 * elements may be fetched, and are dropped), they are written as zeros (y, total,
 * mean, rstd, d_x) and take no part in a gradient. */
typedef struct {
    int32_t dtype;           /* fs_dtype of x, residual, total, y and their gradients */
    int32_t batch, n;        /* >= 0; batch * n <= 2^31 - 1 */
    int32_t width;           /* 1..16384 */
    float eps;               /* >= 0 (0: y of a constant row is not defined: NaN, or what
                                the rounding of its mean leaves) */
    const int32_t* lengths;  /* device [batch], clamped to 0..n; or NULL (n) */
} fs_layer_norm_desc;

/* Bytes of workspace of the backward call (forward needs none); at least 256,
 * or 0 for an invalid desc.  Pure host function. */
size_t fs_layer_norm_workspace_bytes(const fs_layer_norm_desc* desc);

/* residual, total: views, both or neither (data NULL).  weight, bias: device
 * fp32 [width], NULL for ones and for zeros.  mean, rstd: device fp32
 * [batch][n], kept for the backward call, or NULL. */
fs_status fs_layer_norm(const fs_layer_norm_desc* desc, fs_rows x, fs_rows residual,
                        const float* weight, const float* bias, fs_rows total, fs_rows y,
                        float* mean, float* rstd, void* stream);

/* Gradients, given those of y (d_y) and of total (d_total, data NULL: none).
 * z is the forward call's total (x where it had no residual), mean and rstd
 * its statistics.  d_x is the gradient of x and of the residual alike.
 * d_weight, d_bias: device fp32 [width], NULL: not wanted.  All outputs are
 * written, not added to.  workspace: 256-byte aligned. */
fs_status fs_layer_norm_backward(const fs_layer_norm_desc* desc, fs_rows z, const float* weight,
                                 const float* mean, const float* rstd, fs_rows d_y,
                                 fs_rows d_total, fs_rows d_x, float* d_weight, float* d_bias,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* ---- scores of states held in 8-bit integers -----------------------------
 * Rows (tokens) and columns (channels, or the other set's states) each have a
 * scale of their own: x_ik is about scale_i q_ik. */

/* q = 127 x / max |row| to the nearest whole number (ties to the even one, the
 * quotient decided exactly), scale = max |row| / 127.  A row of zeros has scale
 * 0; a row that holds an infinity or a NaN has scale NaN and q = 0, so that all
 * it stands for is NaN.  x: [rows][width] of dtype; q: int8, stride in elements;
 * scale: device fp32 [rows].  0 <= rows < 2^31, 1 <= width <= 65536. */
fs_status fs_quantize_rows(int32_t dtype, int32_t rows, int32_t width, const void* x,
                           int64_t x_stride, int8_t* q, int64_t q_stride, float* scale,
                           void* stream);

/* y[i][j] = scale_x[i] scale_w[j] sum_k q_x[i][k] q_w[j][k] + bias[j].  The sum is
 * exact; it, its product with scale_x and the rest in one are rounded to fp32, y to
 * its type.  q_x: [m][k] and q_w: [n][k] int8 (any value, -128 too), y: [m][n] of
 * dtype; strides of rows in elements.  bias: device fp32 [n] or NULL.  0 <= m, n
 * <= 2^24, m n <= 2^36, 0 <= k <= 65536 (k = 0: the sum is 0).  With more than 32
 * rows an operand whose rows are not 16-byte aligned, or whose k is no multiple of
 * 16, is laid out in the workspace by each call: keep weights aligned. */
typedef struct {
    int32_t dtype; /* fs_dtype of y */
    int32_t m, n, k;
    const int8_t* q_x;
    int64_t q_x_stride;
    const float* scale_x; /* device [m] */
    const int8_t* q_w;
    int64_t q_w_stride;
    const float* scale_w; /* device [n] */
    const float* bias;    /* device [n] or NULL */
    void* y;
    int64_t y_stride;
} fs_quantized_product_desc;

/* Bytes of workspace (from the sizes, the strides and the operands' alignment; q_x or
 * q_w NULL: enough for any address); at least 256, or 0 if the sizes are out of range.
 * Pure host function. */
size_t fs_quantized_product_workspace_bytes(const fs_quantized_product_desc* desc);

fs_status fs_quantized_product(const fs_quantized_product_desc* desc, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ---- distillation of a teacher's top logits -------------------------------
 * Row i has `classes` logits x of the student and k entries (class ids[i][j],
 * logit teacher[i][j]) of a teacher.  With p = softmax(x / T) and, over the
 * entries, tau = softmax(teacher / T), or tau_j = exp(teacher_j / T -
 * teacher_lse[i]) where the teacher's whole row log-sum-exp (of teacher / T) is
 * given (the weights then sum to W < 1, the mass of the entries):
 *   loss_i = T^2 sum_j tau_j (log tau_j - log p[ids_j])
 *   d_logits_ic = d_loss_i T (W p_c - sum_{j: ids_j = c} tau_j).
 * Entries whose class lies outside 0..classes - 1, or whose logit is -inf, are
 * none; a class may be named twice.  Rows with active[i] == 0 are not read,
 * whatever they hold.  Rows without an entry, of -inf alone, or not active have
 * loss 0 and a gradient of zeros; lse of rows that are not active is 0 (of a row
 * of -inf alone: -inf).  Where d_loss is 0 the gradient is zeros.  A class of the
 * teacher's whose logit is -inf makes the loss infinite, not the gradient.  A NaN or
 * +inf among a row's logits makes its lse NaN and, where the row has an entry, its
 * loss and gradient; one among its teacher's logits (or, beside a teacher_lse, one
 * whose quotient by T is too large for fp32) its loss and gradient. */
typedef struct {
    int32_t dtype;            /* fs_dtype of the logits and their gradient */
    int32_t rows;             /* >= 0 */
    int32_t classes;          /* 1..2^24 */
    int32_t k;                /* 1..1024 */
    float temperature;        /* T, in [2^-20, 2^20] */
    const int32_t* ids;       /* device [rows][k] */
    const float* teacher;     /* device [rows][k] */
    const float* teacher_lse; /* device [rows] or NULL */
    const uint8_t* active;    /* device [rows] or NULL */
    /* device fp32 [rows] or NULL: what lse lacks in fp32, written with it and read by
     * the gradient call.  Without it that call's p are off by a factor of up to 1 +
     * 2^-24 |lse| (5e-7 at 8), and T has to be 2^-10 or more; the one call for both
     * never needs it. */
    float* lse_rest;
} fs_distill_desc;

/* Bytes of workspace of fs_distill_loss; at least 256, or 0 for an invalid desc
 * (device pointers are not looked at).  Pure host function. */
size_t fs_distill_workspace_bytes(const fs_distill_desc* desc);

/* loss, lse (log-sum-exp of x / T, kept for the backward call): device fp32
 * [rows].  With d_logits (data not NULL) and d_loss (device fp32 [rows]) the
 * gradient is written by the same call, for a loss whose rows' weights in the
 * total are known beforehand.  workspace: 256-byte aligned. */
fs_status fs_distill_loss(const fs_distill_desc* desc, fs_rows logits, float* loss, float* lse,
                          const float* d_loss, fs_rows d_logits, void* workspace,
                          size_t workspace_bytes, void* stream);

/* The gradient alone, given the forward call's lse. */
fs_status fs_distill_loss_backward(const fs_distill_desc* desc, fs_rows logits, const float* lse,
                                   const float* d_loss, fs_rows d_logits, void* stream);

/* ---- balanced use of the columns -------------------------------------------
 * Each row of `experts` logits chooses its k largest columns (ties: the lowest
 * column; NaN counts as -inf); with p = softmax(logits), for each batch entry,
 * its N rows that take part, c_e the number of rows that chose column e:
 *   loss[b][0] = experts sum_e (c_e / (k N)) (mean_i p_ie),
 *   loss[b][1] = mean_i lse_i^2,
 *   gates_ij = p[ids_ij], over the row's sum of them if normalize.
 * Rows i >= lengths[b] (padding: nothing depends on what they hold, though a first
 * few elements may be fetched) and rows of -inf alone take no part: ids -1, gates
 * and lse 0.  Where no row takes part the losses are 0.  The columns chosen have no
 * gradient.  A NaN or +inf among a row's logits (or a row of NaN alone) makes its
 * gates, lse and gradient NaN, and its batch entry's losses. */
typedef struct {
    int32_t dtype;           /* fs_dtype of the logits and their gradient */
    int32_t batch, n;        /* >= 0; batch <= 65535, batch * n and n * k <= 2^31 - 1 */
    int32_t experts;         /* 1..1024 */
    int32_t k;               /* 1..min(32, experts) */
    int32_t normalize;
    const int32_t* lengths;  /* device [batch], clamped to 0..n; or NULL (n) */
} fs_balance_desc;

/* Bytes of workspace of fs_balance_loss; at least 256, or 0 for an invalid desc.
 * Pure host function. */
size_t fs_balance_workspace_bytes(const fs_balance_desc* desc);

/* ids: int32 [batch][n][k], largest first; gates: fp32 [batch][n][k]; counts: int32
 * [batch][experts]; loss: fp32 [batch][2]; lse: fp32 [batch][n] (all device,
 * written).  workspace: 256-byte aligned. */
fs_status fs_balance_loss(const fs_balance_desc* desc, fs_rows logits, int32_t* ids, float* gates,
                          int32_t* counts, float* loss, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Gradient of the logits, given those of loss (d_loss, [batch][2]) and of gates
 * (d_gates, [batch][n][k], or NULL for none); ids, counts and lse are the
 * forward call's (ids and counts may also come from another choice, such as a
 * plan's: counts then hold k for each row that takes part, a row whose first
 * id is negative takes none, and other ids out of range are no choice). */
fs_status fs_balance_loss_backward(const fs_balance_desc* desc, fs_rows logits, const int32_t* ids,
                                   const int32_t* counts, const float* lse, const float* d_loss,
                                   const float* d_gates, fs_rows d_logits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FS_LAYERS_H */

/*
 * fs_attention.h -- C ABI of the row-normalised attention between two sets of
 * states, its gradients, and the preparation of its queries and keys, on AMD
 * MI355X (gfx950).  Part of libfs_sinkhorn.so; status codes, stream and error
 * conventions are those of fs_sinkhorn.h.
 *
 * The solver's f-update is a row log-sum-exp of a biased score matrix between
 * two clouds and its transport the weighted average that goes with it.  These
 * entry points are the ordinary form of that traversal for the features a
 * model forms before (or after) it matches the two sets: many heads, batches
 * of ragged lengths, masks, 16-bit types, a learned bias, and gradients with
 * respect to everything learned.  The score matrix never reaches memory here
 * either.
 *
 * Conventions (every entry point of this file):
 *  - Tensors are device memory on the calling thread's current device, of
 *    element type `dtype`, given as fs_rows: a [batch][rows][heads][width]
 *    view whose last axis is contiguous and whose other strides (in elements)
 *    are free, so both [b][row][head][w] and [b][head][row][w] layouts, slices
 *    of a fused projection, and inputs broadcast by stride 0 are fine.  Views
 *    whose rows are 16-byte aligned with a width of whole 16-byte chunks are
 *    read with wide loads, others element by element.  Outputs may not overlap
 *    themselves, one another, an input or the workspace (slices of one buffer
 *    side by side do not overlap; against an input whole extents count).
 *  - Work is enqueued on `stream` and is asynchronous; nothing synchronises,
 *    nothing is allocated, and every call may be captured into a graph (a
 *    replay uses the same buffers: two captured calls that may overlap need a
 *    workspace each).  Equal calls give equal bits: no sum depends on the
 *    order in which workgroups run.
 *  - Sums, softmax statistics and norms are fp32 (sums over workgroups' parts of
 *    a weight's or a bias's gradient in 64 bits).  In a 16-bit type the weights P
 *    and dS are rounded to that type before their products with v, d_o, q and k,
 *    as the matrix units take them; an output is rounded once more.  Against the
 *    definition in 64 bits that gives about 1.4 times the error of a product in
 *    fp32 rounded once (bf16: 0.0023 against 0.0017 relative).
 *  - A launch has fewer than 2^32 threads: batch * heads may reach about 2^23 with
 *    few rows, and batch * heads * rows 2^31; more is refused.
 */
#ifndef FS_ATTENTION_H
#define FS_ATTENTION_H

#include "fs_sinkhorn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FS_DTYPE_F32 = 0, FS_DTYPE_BF16 = 1, FS_DTYPE_F16 = 2 } fs_dtype;

/* A [batch][rows][heads][width] view; strides in elements, >= 0. */
typedef struct {
    void* data;
    int64_t stride_batch, stride_row, stride_head;
} fs_rows;

/* What one attention call computes.  For batch entry b, query row i < n, key
 * row j < m, head h, with key head h / (heads / kv_heads):
 *   s_ij = scale q_i.k_j + bias[bucket(j - i - offset_b)][h]
 *   L_i  = log sum_j exp(s_ij)          (lse, [batch][heads][n] fp32)
 *   O_i  = sum_j exp(s_ij - L_i) v_j
 * over the visible keys: j < kv_len[b], key_mask[b][j] != 0 and, if causal,
 * j <= i + offset_b.  Rows i >= q_len[b] and rows without a visible key give
 * O = 0 and L = -inf and take part in no gradient.  Not used, whatever they hold
 * (NaN, infinities): q, d_o and d_lse of such rows (but q of a row that only the
 * bias empties), and k and v of keys that no row sees.  A key that some row sees
 * is read for the rows around it too: if it holds NaN, they may. */
typedef struct {
    int32_t dtype;            /* fs_dtype of q, k, v, o and their gradients */
    int32_t batch, n, m;      /* >= 0; n, m <= 2^28 */
    int32_t heads, kv_heads;  /* >= 1, heads a multiple of kv_heads and <= 65535 */
    int32_t d, dv;            /* widths of q, k and of v, o: 1..256 (fp32: 1..128) */
    float scale;              /* > 0, <= 2e38 */
    int32_t causal;
    int32_t offset;           /* position of query row 0 among the keys, |.| <= 2^29 */
    const int32_t* offsets;   /* device [batch], in place of offset; or NULL */
    const int32_t* q_len;     /* device [batch] or NULL (n); clamped to 0..n */
    const int32_t* kv_len;    /* device [batch] or NULL (m); clamped to 0..m */
    const uint8_t* key_mask;  /* device [batch][key_mask_stride], 0 = hidden; or NULL */
    int64_t key_mask_stride;  /* elements; >= 0 */
    /* Learned bias by buckets of the relative position r = j - i - offset_b.
     * edges: host array, ascending, each 1..1024, read during the call.  With
     * u(x) = the number of edges <= x, the bucket is u(max(-r, 0)) one-sided
     * (n_edges + 1 buckets: keys after the query count as distance 0), or
     * two-sided u(|r|) for r <= 0 and n_edges + 1 + u(r) for r > 0
     * (2 (n_edges + 1) buckets).  bias: device fp32 [buckets][heads], or NULL
     * for none.  An entry of -1e6 or less gives its pairs no weight, as a mask (a
     * row that has no other pairs is empty); the others are at most 1e6 (fp32 holds
     * few of a score's digits beside it).  The bias speaks of positions: it is for rows and
     * keys that have an order, such as points along a curve or a scan. */
    const float* bias;
    const int32_t* edges;
    int32_t n_edges;          /* 0..255 */
    int32_t two_sided;
} fs_attention_desc;

/* Edges of `side_buckets` buckets on one side: one distance each for the first
 * half, the rest evenly spaced in the logarithm up to max_distance, each edge
 * the smallest whole number not below the exact value (whole-number
 * arithmetic).  Writes side_buckets - 1 edges.  2 <= side_buckets <= 64,
 * side_buckets / 2 < max_distance <= 1024.  Pure host function. */
fs_status fs_bucket_edges(int32_t side_buckets, int32_t max_distance, int32_t* edges);

/* Bytes of workspace for the forward (backward == 0) or backward call (the
 * larger of both serves both); at least 256, or 0 for an invalid desc.  Device
 * pointers of desc are only tested against NULL.  Pure host function. */
size_t fs_attention_workspace_bytes(const fs_attention_desc* desc, int32_t backward);

/* o (written) and, unless NULL, lse (written, [batch][heads][n] contiguous).
 * Work: with many query rows, workgroups of 128 rows stream the keys once per
 * head; with few (single tokens, or a small problem) the rows of all heads of
 * a key head share a pass over the keys.  Where workgroups are few, the keys
 * are split over them and joined in a fixed order.  workspace: 256-byte
 * aligned. */
fs_status fs_attention_forward(const fs_attention_desc* desc, fs_rows q, fs_rows k, fs_rows v,
                               fs_rows o, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Gradients, given those of o (d_o) and of lse (d_lse, [batch][heads][n]
 * contiguous fp32, or NULL for none).  o and lse are the forward call's.  d_q,
 * d_k, d_v (views; data NULL: not wanted) and d_bias (device fp32
 * [buckets][heads]; NULL: not wanted) are written, not added to.  d_k and d_v
 * are summed over the query heads that share a key head.  For an input that
 * was broadcast by a stride of 0 each copy's gradient is written (the
 * caller's to sum).  The rows' sums of P dP are formed in fp32 by the pass that
 * writes d_q (run for d_bias too); d_k and d_v asked for without either take
 * them from the stored, rounded o. */
fs_status fs_attention_backward(const fs_attention_desc* desc, fs_rows q, fs_rows k, fs_rows v,
                                fs_rows o, const float* lse, fs_rows d_o, const float* d_lse,
                                fs_rows d_q, fs_rows d_k, fs_rows d_v, float* d_bias,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Preparation of queries and keys: the norm of every head's row and the
 * rotation by its position, both tensors in one launch (the counterpart of
 * the normalisation that the cosine cost does to its points):
 *   z = weight x / sqrt(mean(x^2) + eps),   y = R(position) z,
 * where R turns pair p < rot / 2 by the angle whose cosine and sine are
 * cos_table[position][p], sin_table[position][p]; the pair is the elements
 * (p, p + rot / 2), or (2 p, 2 p + 1) if interleaved; elements from rot on are
 * not turned.  Either q or k may be left out (heads 0). */
typedef struct {
    int32_t dtype;               /* fs_dtype of x and y */
    int32_t batch, n;            /* >= 0, batch * n <= 2^26 */
    int32_t heads_q, heads_k;    /* >= 0, either may be 0; batch * n * their sum <= 2^31 */
    int32_t d;                   /* 2..256, even */
    int32_t rot;                 /* 0..d, even; 0: no rotation */
    int32_t interleaved;
    float eps;                   /* >= 0 (0: a row of zeros gives NaN) */
    const float* cos_table;      /* device fp32 [n_pos][rot / 2] (NULL if rot == 0) */
    const float* sin_table;
    int32_t n_pos;               /* >= 1 if rot > 0 */
    const int32_t* positions;    /* device [batch][positions_stride], or NULL: row i stands at
                                    offset + i; clamped to 0..n_pos - 1 */
    int64_t positions_stride;    /* elements; >= 0 */
    int32_t offset;
} fs_qk_norm_desc;

/* Bytes of workspace of the backward call (forward needs none); at least 256,
 * or 0 for an invalid desc.  Pure host function. */
size_t fs_qk_norm_workspace_bytes(const fs_qk_norm_desc* desc);

/* q_weight, k_weight: device fp32 [d], or NULL for ones. */
fs_status fs_qk_norm_rotate(const fs_qk_norm_desc* desc, fs_rows q, fs_rows k,
                            const float* q_weight, const float* k_weight, fs_rows q_out,
                            fs_rows k_out, void* stream);

/* Gradients with respect to q, k and the weights, given those of q_out and
 * k_out; q, k are the forward call's inputs.  d_q_weight, d_k_weight: device
 * fp32 [d], NULL: not wanted.  All outputs are written, not added to.
 * workspace: 256-byte aligned. */
fs_status fs_qk_norm_rotate_backward(const fs_qk_norm_desc* desc, fs_rows q, fs_rows k,
                                     const float* q_weight, const float* k_weight,
                                     fs_rows d_q_out, fs_rows d_k_out, fs_rows d_q, fs_rows d_k,
                                     float* d_q_weight, float* d_k_weight, void* workspace,
                                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FS_ATTENTION_H */

/*
 * moe_rows.h -- C ABI of the layer's row operators: token rows to expert order and
 * back with their gradients, and products of rows in 8-bit integers.  Implemented by
 * the same library as moe.h, whose conventions hold here except where a section says
 * otherwise.
 */
#ifndef MOE_B200_ROWS_H
#define MOE_B200_ROWS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rows
 * Token rows to expert order and back, with their gradients, for programs that
 * run the experts (or train them) themselves.  With inv [T, k] the inverse of
 * the expert order (inv[t, j] = the expert-order row of token t's slot j, or
 * MOE_NOT_ROUTED), n = T * k and s = dims->routed_scaling_factor:
 *
 *   moe_sort               counts, offsets, perm and inv (optionally moe_dispatch too)
 *   moe_dispatch           x_perm[inv[t, j]] = x[t]
 *   moe_dispatch_backward  d_x[t] = sum_j d_x_perm[inv[t, j]] + add[t]
 *   moe_combine            y[t] = s * sum_j topk_w[t, j] * o[inv[t, j]] + shared[t]
 *   moe_combine_backward   d_o[inv[t, j]] = s * topk_w[t, j] * d_y[t]
 *                          d_topk_w[t, j] = s * <d_y[t], o[inv[t, j]]>
 *                          (the gradient of `shared` is d_y itself)
 *   moe_route_backward     d_logits from d_topk_w, through the normalisation and the sigmoid
 *
 * Conventions of these calls, where they differ from the ones above:
 * - dims supplies T, d_model, num_experts, num_experts_per_tok,
 *   routed_scaling_factor and norm_topk_prob; any d_model from 1 to 2^30 (the
 *   widths F and Fs and the flags are ignored).  E <= 512, k <= min(E, 16) hold;
 *   T * k <= 2^31 - 4097.
 * - Row matrices are bf16, fp16 or fp32 (moe_dtype) with a row stride in
 *   elements (>= d_model); 16-byte-aligned bases.  Rows whose stride is no
 *   multiple of 16 bytes are taken, more slowly.
 * - T = 0 (rows = 0, M = 0 below) returns MOE_OK with any pointers.
 * - Slots that are not routed are skipped: they add nothing, and their entry
 *   of d_topk_w is 0.  Expert-order rows that no slot names (behind the last
 *   routed row) are neither read nor written.  A token without experts gets
 *   y = shared (0 without), d_x = add (0 without) and zero d_logits.
 * - Sums run in fp32 in slot order and are rounded once; the results do not
 *   depend on the launch.
 * - ws is optional (NULL), or a 256-byte status header (256-byte aligned; a
 *   workspace starts with one): an inv entry outside [-1, n) or an expert id
 *   outside [-1, E) is skipped and recorded there as MOE_ERR_DEVICE_BOUNDS.
 *   These calls do not clear the status word (moe_sort, moe_route, moe_permute
 *   and moe_forward do), so one moe_read_device_status after a run of them
 *   reports the first error of the run. */
typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F16 = 1, MOE_DTYPE_F32 = 2 } moe_dtype;

/* Bytes of workspace that moe_sort needs for every batch of up to dims->T tokens
 * (0 if the dims are invalid; never less for more tokens).  For one batch, any
 * workspace of moe_workspace_size for its T, E and k is large enough. */
size_t moe_sort_workspace_size(const moe_dims_t *dims);

/* moe_permute with the inverse permutation inv [T, k], and rows of any
 * moe_dtype and stride: if x and x_perm are both non-NULL, moe_dispatch follows
 * in the same call.  Clears the status word first.  T = 0 sets counts and
 * offsets to zero. */
moe_status moe_sort(const moe_dims_t *dims, const int32_t *topk_idx, int32_t *counts,
                    int32_t *offsets, int32_t *perm, int32_t *inv, int32_t dtype, const void *x,
                    int64_t x_stride, void *x_perm, int64_t x_perm_stride, void *ws,
                    size_t ws_bytes, void *stream);

/* x [T, d] -> x_perm [T * k, d], the same type. */
moe_status moe_dispatch(const moe_dims_t *dims, int32_t dtype, const void *x, int64_t x_stride,
                        const int32_t *inv, void *x_perm, int64_t x_perm_stride, void *ws,
                        void *stream);

/* d_x_perm [T * k, d] and add [T, d] (NULL = none) of in_dtype -> d_x [T, d] of
 * out_dtype.  d_x may be add itself (MOE_ERR_INVALID_ARG then unless type and stride
 * are the same). */
moe_status moe_dispatch_backward(const moe_dims_t *dims, int32_t in_dtype, const void *d_x_perm,
                                 int64_t d_x_perm_stride, const int32_t *inv, const void *add,
                                 int64_t add_stride, int32_t out_dtype, void *d_x,
                                 int64_t d_x_stride, void *ws, void *stream);

/* o [T * k, d] and shared [T, d] (NULL = none) of in_dtype, topk_w [T, k] fp32 ->
 * y [T, d] of out_dtype.  y may be shared itself (MOE_ERR_INVALID_ARG then unless type
 * and stride are the same). */
moe_status moe_combine(const moe_dims_t *dims, int32_t in_dtype, const void *o, int64_t o_stride,
                       const int32_t *inv, const float *topk_w, const void *shared,
                       int64_t shared_stride, int32_t out_dtype, void *y, int64_t y_stride,
                       void *ws, void *stream);

/* d_y [T, d], o [T * k, d] -> d_o [T * k, d] of the same type, d_topk_w [T, k]
 * fp32.  d_o may be o itself (same stride): the gradient then replaces the
 * rows it was computed from. */
moe_status moe_combine_backward(const moe_dims_t *dims, int32_t dtype, const void *d_y,
                                int64_t d_y_stride, const void *o, int64_t o_stride,
                                const int32_t *inv, const float *topk_w, void *d_o,
                                int64_t d_o_stride, float *d_topk_w, void *ws, void *stream);

/* Gradient of the router's logits [T, E] (fp32, as moe_logits_offset finds them,
 * the logit bias included) from that of its weights: with s_j = sigmoid(l_j) over
 * a token's selected experts and p_j = s_j / sum_i s_i,
 *   norm_topk_prob:  d_l_j = p_j * (1 - s_j) * (d_w_j - sum_i d_w_i * p_i)
 *   without:         d_l_j = s_j * (1 - s_j) * d_w_j
 * d_logits [T, E] is written whole: zero for experts that were not selected.
 * An expert that a row names more than once gets the sum of its slots. */
moe_status moe_route_backward(const moe_dims_t *dims, const float *logits, const int32_t *topk_idx,
                              const float *d_topk_w, float *d_logits, void *ws, void *stream);

/* ------------------------------------------------------------------ 8-bit integers
 * Rows quantized to int8 with one fp32 scale each, and products of such rows:
 * the scale of a token (row of activations) and of a channel (row of weights).
 *   s = max(amax(|row|) / 127, 2^-126)  (1 for a row of zeros),
 *   code = rint(v * (1 / s))
 * every step one correctly rounded fp32 operation, ties to even, as
 * moe_prepare_fp8 does for e4m3.  A row that holds an infinity or NaN gets the
 * scale NaN and codes 0, so that every product of it is NaN. */

/* x [rows, cols] (cols <= 2^30) of `dtype` (row stride in elements) -> codes (row stride in
 * bytes, a multiple of 16; the bytes past cols are not written) and scales
 * [rows].  n_rows (device, NULL = rows): only the first *n_rows rows are
 * quantized, the others left as they were. */
moe_status moe_quantize_int8(int32_t rows, int32_t cols, int32_t dtype, const void *x,
                             int64_t x_stride, const int32_t *n_rows, int8_t *codes,
                             int64_t codes_stride, float *scales, void *stream);

/* moe_dispatch of quantized rows: the codes and the scale of x[t], computed once,
 * are stored to row inv[t, j] of codes [T * k, d] and scales [T * k]. */
moe_status moe_dispatch_int8(const moe_dims_t *dims, int32_t dtype, const void *x,
                             int64_t x_stride, const int32_t *inv, int8_t *codes,
                             int64_t codes_stride, float *scales, void *ws, void *stream);

/* moe_int8_matmul_t flags: out = silu(gate) * up, where b holds 2 N rows per group:
 * the N gate channels, then the N up channels.  silu is off by at most about 5 + 1.2 |gate|
 * units in the last place of fp32 for gate < 0 (a few for gate > 0), and is 0 below -87. */
#define MOE_INT8_SWIGLU 1

/* out[r, c] = (sum_k a[r, k] * b[g, c, k]) * a_scale[r] * b_scale[g, c] for the rows
 * r of group g: rows offsets[g] to offsets[g + 1] - 1 (expert order; a device
 * array), or all M rows where offsets is NULL and G = 1.  The integer sums are
 * exact.  Rows outside every group are not written.  Offsets that decrease or
 * leave [0, M] are clamped and recorded as MOE_ERR_DEVICE_BOUNDS, and so is an
 * infinite result in fp16 output (one beyond the type's range).
 * a: [M, K] int8, b: [G * N, K] int8 (2 N rows per group with MOE_INT8_SWIGLU), row
 * strides in bytes, multiples of 16; out: [M, N] of out_dtype, row stride in
 * elements.  Any N; K <= 131071; G <= 512.  ws needs only 256 bytes (status
 * header; not cleared by this call). */
typedef struct {
    uint32_t struct_size;   /* sizeof(moe_int8_matmul_t) */
    int32_t M, N, K, G;
    int32_t out_dtype;      /* moe_dtype */
    int32_t flags;          /* MOE_INT8_* */
    const int8_t *a;
    int64_t a_stride;
    const float *a_scale;   /* [M] */
    const int8_t *b;
    int64_t b_stride;
    const float *b_scale;   /* one per row of b */
    const int32_t *offsets; /* [G + 1] device, or NULL */
    void *out;
    int64_t out_stride;
} moe_int8_matmul_t;

moe_status moe_matmul_int8(const moe_int8_matmul_t *args, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* MOE_B200_ROWS_H */

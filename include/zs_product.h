/*
 * zs_product.h - matrix products exported by libzs.so beside the activation operators (zs_act.h):
 * a linear layer's products with an 8-bit weight, the experts' products over groups of rows with
 * their weight gradients, and the way of tokens to their experts and back.
 *
 * An 8-bit checkpoint (zs_act) that zs_rmsnorm has written is the input of zs_product8 as it is,
 * and zs_expert_wgrad leaves the experts' gradients in the contiguous gradient buffer that the
 * step reads ("Deep dive: Megatron", section "Distributed optimizer").
 *
 * An 8-bit weight (outs x cols, of a layer y = x W^T) holds
 *   codes:   outs x Pc bytes, Pc = cols rounded up to a multiple of 128; e4m3 (1 sign, 4 exponent,
 *            3 mantissa bits); the Pc - cols codes behind each row are zero;
 *   codes_t: NULL, or cols x Po bytes, Po = outs rounded up to a multiple of 128: the same codes
 *            transposed, what the input's gradient dy W reads; the Po - outs behind each row are
 *            zero;
 *   scales:  (Po / 128) x (Pc / 128) bytes, one per block of 128 x 128: the biased exponent b of a
 *            power-of-two scale s = 2^(b - 127).
 * An element's value is code * s; s and the codes follow zs_act's rule for ZS_E4M3, over the
 * block's elements: nothing is clipped, a block with an infinity or a NaN has b = 255 and stands
 * for NaN throughout.  A square block serves both orientations with the same codes.
 *
 * Conventions as in zs.h and zs_act.h, and:
 *   - rows, cols, outs and experts may be any number within the limits; a matrix of no rows is
 *     written as such.  Matrices at any row stride and alignment of their elements give the same
 *     results; those with a base, row stride and expert stride of a multiple of 4 bytes run fastest
 *     (where rows of a matrix run along the sum, as those of w do with in_major and those of x and
 *     dy in the weight gradient, with a multiple of 8 columns too).
 *   - an output may not lie in an input's memory, but where a call says so; one that begins where an
 *     input does is refused.
 *   - ends: device memory, one int32 per expert: the row behind its last; its first row is the one
 *     behind the expert's before it (0 for the first).  The kernels read them when they run.  An
 *     end counts as the largest one up to it, within 0 .. rows, so that no value leads out of the
 *     matrices.
 */
#ifndef ZS_PRODUCT_H
#define ZS_PRODUCT_H

#include <stdint.h>

#include "zs_act.h"

#ifdef __cplusplus
extern "C" {
#endif

/* An 8-bit weight's arrays (device memory, 16-byte aligned but for scales). */
typedef struct {
    void* codes;
    void* codes_t; /* or NULL */
    void* scales;
} zs_weight8;

/* Bytes of the arrays of an outs x cols weight.  Host only.
 * Errors: ZS_EINVAL on a NULL output, outs or cols outside 1 .. 2^23 or sizes past one launch. */
zs_status zs_weight8_size(int64_t outs, int64_t cols, int64_t* codes_bytes, int64_t* codes_t_bytes,
                          int64_t* scales_bytes);

/* Write the 8-bit form of src (outs x cols, bf16, fp16 or fp32), the transposed codes too if
 * w8->codes_t is not NULL.
 * Errors: ZS_EINVAL on a NULL pointer, a bad dtype, size, stride or alignment. */
zs_status zs_weight8_pack(const void* src, zs_dtype src_dtype, int64_t src_stride, int64_t outs, int64_t cols,
                          const zs_weight8* w8, void* stream);

/* Product of an 8-bit checkpoint (ZS_E4M3) and an 8-bit weight:
 *   transposed 0:  y[r][n] = sum over k of x8[r][k] * w8[n][k]    x8: rows x cols, y: rows x outs
 *   otherwise:     y[r][k] = sum over n of x8[r][n] * w8[n][k]    x8: rows x outs, y: rows x cols
 * (the second takes codes_t: the input's gradient from that of the output, in 8 bits).  Products
 * are summed in fp32 on the matrix cores, which align the products of eight consecutive elements
 * to the largest of them and cut off what lies 2^-13 below; the result is rounded once to y_dtype,
 * bf16 or fp16.  A checkpoint with one scale per 128 columns is one whose four scale bytes of
 * those columns are equal.  A row of x8 with a NaN is NaN throughout, and so is a column of y
 * whose weights hold one.
 * Errors: ZS_EINVAL on a NULL pointer, a bad dtype, size, stride or alignment, a checkpoint in
 * ZS_INT8, or a missing codes_t. */
zs_status zs_product8(const zs_act* x8, int64_t rows, const zs_weight8* w8, int64_t outs, int64_t cols,
                      int32_t transposed, void* y, zs_dtype y_dtype, int64_t y_stride, void* stream);

/* Products of groups of rows with their expert's weight: for each row r of expert e
 *   y[r] = x[r] W_e^T   with W_e outs x cols, or
 *   y[r] = x[r] W_e     with W_e cols x outs, when in_major is not 0
 *   x: rows x cols;  y: rows x outs;  dtype: bf16 or fp16 for all three.
 *   w: the experts' matrices, w_expert_stride elements apart.
 *   zero_rest: not 0 writes zeros into the rows of y behind the last expert's; 0 leaves them.
 * Summed in fp32, rounded once.  rows is at most 2^31 - 4096, experts 1 .. 1024.
 * Errors: ZS_EINVAL on a NULL pointer, a bad dtype, size, stride or alignment, or sizes past one
 * launch. */
zs_status zs_expert_product(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                            int64_t w_expert_stride, zs_dtype dtype, const int32_t* ends, int32_t experts,
                            int64_t rows, int64_t cols, int64_t outs, int32_t in_major, void* y, int64_t y_stride,
                            int32_t zero_rest, void* stream);

/* Weight gradients of the experts: dw_e = base_e + sum over the rows r of expert e of dy[r]^T x[r].
 *   x: rows x cols, dy: rows x outs, of dtype bf16 or fp16.
 *   dw: for each expert outs x cols, or cols x outs when in_major is not 0, dw_expert_stride
 *       elements apart, of dw_dtype (dtype or fp32): a view of the flat gradient buffer, for
 *       instance.  base: NULL or a matrix of the same type and strides; dw itself adds to what is
 *       there.  An expert without rows gets its base, or zeros.
 * Summed in fp32 in a fixed order, rounded once.
 * Errors: as zs_expert_product, and ZS_EINVAL for experts' matrices that overlap; ZS_EUNSUPPORTED
 * for a dw_dtype that is neither dtype nor fp32. */
zs_status zs_expert_wgrad(const void* x, int64_t x_stride, const void* dy, int64_t dy_stride, zs_dtype dtype,
                          const int32_t* ends, int32_t experts, int64_t rows, int64_t cols, int64_t outs, void* dw,
                          zs_dtype dw_dtype, int64_t dw_stride, int64_t dw_expert_stride, int32_t in_major,
                          const void* base, void* stream);

/* Bytes of zs_route's workspace (at least 16).  Host only.
 * Errors: ZS_EINVAL on a NULL output, slots outside 0 .. 2^31 - 4096 or experts outside 1 .. 1024. */
zs_status zs_route_workspace(int64_t slots, int32_t experts, int64_t* bytes);

/* The order of `slots` choices by expert.  Choice s (token s / choices, its choice s % choices)
 * names expert ids[s]; a number outside 0 .. experts - 1 names none.
 *   ids: int32 or int64 (id_bytes 4 or 8).
 *   ends: experts int32: the row behind each expert's last.
 *   slot: slots int32: the choice that row p holds; choices keep their order within an expert.
 *         Rows behind the last expert's hold the choices s that name no expert, as -1 - s.
 *   place: slots int32: the row of each choice, -1 for none.
 *   workspace: device memory of at least zs_route_workspace bytes, 16-byte aligned.
 * Errors: ZS_EINVAL on a NULL pointer, a bad size or alignment, or a missing or small workspace. */
zs_status zs_route(const void* ids, int32_t id_bytes, int64_t slots, int32_t experts, int32_t* ends, int32_t* slot,
                   int32_t* place, void* workspace, int64_t workspace_bytes, void* stream);

/* Rows in the order of their experts: out[p] = x[slot[p] / choices], zeros where slot[p] is not
 * within 0 .. tokens * choices - 1.
 *   x: tokens x cols, out: tokens * choices x cols, of dtype bf16, fp16 or fp32.
 * tokens * choices is at most 2^31 - 4096, and the rows of out, at 16 lanes to a row of up to 256 bytes
 * and twice as many up to each power of two, but 256 at most, have fewer than 2^32 lanes: that is
 * below 2^28 rows of up to 256 bytes and 2^24 of more than 2048.
 * Errors: ZS_EINVAL on a NULL pointer, a bad dtype, size, stride or alignment, or sizes past one launch. */
zs_status zs_expert_gather(const void* x, int64_t x_stride, zs_dtype dtype, const int32_t* slot, int64_t tokens,
                           int32_t choices, int64_t cols, void* out, int64_t out_stride, void* stream);

/* Rows back to their tokens: out[t] = sum over j of weights[t][j] * y[place[t][j]] in order of j, in
 * fp32, rounded once.  Choices whose place is not within 0 .. tokens * choices - 1 count nothing.
 *   y: tokens * choices x cols, out: tokens x cols, of dtype bf16, fp16 or fp32.
 *   weights: NULL (ones) or tokens x choices fp32, consecutive.
 * Errors: as zs_expert_gather, whose limits hold for the tokens here. */
zs_status zs_expert_combine(const void* y, int64_t y_stride, zs_dtype dtype, const int32_t* place,
                            const float* weights, int64_t tokens, int32_t choices, int64_t cols, void* out,
                            int64_t out_stride, void* stream);

/* Backward pass of zs_expert_combine, for each token t and its choice j in row p = place[t][j]:
 *   dy[p] = weights[t][j] * dout[t];  dweights[t][j] = sum over columns of dout[t] * y[p], in fp32.
 * A choice whose place is not within 0 .. tokens * choices - 1 has the weight gradient 0; a row p with
 * slot[p] < 0 gets zeros.  (With zs_route's slot and place every row of dy is written; a place that
 * two choices share, which no route has, gets one of the two.)
 *   dy: NULL or a matrix like y.  dweights: NULL or tokens x choices fp32; needs y, which may be
 *   NULL otherwise.  dy may be y itself (same stride).
 * Errors: as zs_expert_combine, and ZS_EINVAL when neither output is given or dy is in y's place at
 * another stride. */
zs_status zs_expert_combine_backward(const void* dout, int64_t dout_stride, const void* y, int64_t y_stride,
                                     zs_dtype dtype, const int32_t* slot, const int32_t* place,
                                     const float* weights, int64_t tokens, int32_t choices, int64_t cols, void* dy,
                                     int64_t dy_stride, float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_PRODUCT_H */

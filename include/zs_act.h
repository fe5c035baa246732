/*
 * zs_act.h - activation operators exported by libzs.so beside the optimizer step (zs.h):
 * 8-bit activation checkpoints, the root-mean-square norm that writes them, its backward
 * pass, and the weight gradient taken from a checkpoint straight into a gradient buffer.
 *
 * Sharding leaves the activations of a rank as they are ("3.7 Megatron-LM, DeepSpeed &
 * Parallelism in Practice", section "ZeRO Stages Recap"), and backward fills the contiguous
 * gradient buffer that the step reads ("Deep dive: Megatron", section "Distributed
 * optimizer").  These calls keep what backward needs at 1.03 bytes per element, and write
 * the gradients where zs_step_flat, zs_pack or zs_unscale_check expects them.
 *
 * A checkpoint of a rows x cols matrix (rows: tokens, cols: features) holds
 *   codes:  rows x P bytes, P = cols rounded up to a multiple of 32, 16-byte aligned; the
 *           P - cols codes behind each row are zero;
 *   scales: rows x (P / 32) bytes, one per 32 consecutive columns of a row: the biased
 *           exponent b of a power-of-two scale s = 2^(b - 127).
 * An element's value is code * s.  s is the smallest power of two (at least 2^-127) with
 * max|x| <= qmax * s over the 32 elements, qmax = 448 (ZS_E4M3: 1 sign, 4 exponent, 3
 * mantissa bits, no infinities) or 127 (ZS_INT8: two's complement), and the code is x / s
 * rounded to nearest, ties to even: nothing is clipped.  A group of zeros has b = 0.  A
 * group with an infinity or a NaN has b = 255 and stands for NaN throughout, so that it
 * reaches the overflow check of the step.  A power of two loses nothing more on the way
 * back: code * s is exact in bf16 and fp32 down to their smallest normal numbers, and in
 * fp16 if the source held fp16 numbers.  Other values are rounded to fp16 once, to nearest
 * even: those of zs_rmsnorm's y8, which is taken before y is rounded, can lie below fp16's
 * smallest step, and those of a bf16 or fp32 source anywhere.  Past fp16's range a value
 * becomes its largest number, not an infinity: the code's rounding can lift an fp16 source
 * there, but a bf16 or fp32 source that really held such a value is cut off in silence.
 *
 * Conventions as in zs.h, and:
 *   - A matrix argument is a device pointer with a row stride in elements (>= cols, or any
 *     value when rows <= 1); columns are consecutive.  Data need no alignment beyond their
 *     element size, except codes (16 bytes) and workspaces (16 bytes).
 *   - Every call works on the current HIP device, which must own all its arrays, and only
 *     enqueues kernels on `stream`: nothing is allocated and the host never waits, so
 *     calls may be captured into a graph.  A workspace is the caller's and is overwritten:
 *     two calls (or graphs) that may overlap need one each.  Its contents mean nothing
 *     afterwards.
 *   - rows may be 0: matrix outputs are then empty, and weight gradients are the base or 0.
 *   - Unless stated otherwise outputs must not overlap inputs or one another.
 *   - Results are the same from call to call: no sum depends on the order in which
 *     workgroups run.
 */
#ifndef ZS_ACT_H
#define ZS_ACT_H

#include <stdint.h>

#include "zs.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ZS_E4M3 = 0, ZS_INT8 = 1 } zs_code;

/* A checkpoint's arrays (device memory) and code; rows and cols go with each call. */
typedef struct {
    void* codes;
    void* scales;
    int32_t code;     /* zs_code */
    int32_t reserved; /* 0 (anything else is ZS_EINVAL) */
} zs_act;

/* Bytes of the codes and scales arrays of a rows x cols checkpoint.  Host only.
 * Errors: ZS_EINVAL on a NULL output, rows < 0, cols < 1 or a size above 2^62. */
zs_status zs_act_size(int64_t rows, int64_t cols, int64_t* codes_bytes, int64_t* scales_bytes);

/* Write the checkpoint of src (bf16, fp16 or fp32).
 * Errors: ZS_EINVAL on a NULL pointer, a bad dtype, code, size, stride or alignment. */
zs_status zs_act_pack(const void* src, zs_dtype src_dtype, int64_t src_stride, int64_t rows, int64_t cols,
                      const zs_act* act, void* stream);

/* Read a checkpoint back into dst (bf16, fp16 or fp32), each value rounded once, to nearest
 * even.  Errors: as zs_act_pack. */
zs_status zs_act_unpack(const zs_act* act, int64_t rows, int64_t cols, void* dst, zs_dtype dst_dtype,
                        int64_t dst_stride, void* stream);

/* Root-mean-square norm of each row, with the addition of the residual before it:
 *   h = x + residual (rounded once to dtype; h = x without a residual)
 *   rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * weight
 * in one pass: x and residual are read once.  The sum of squares is taken in fp64, the rest in
 * fp32, each output rounded once.
 *   x, residual (NULL: none), weight (cols elements): dtype bf16 or fp16.
 *   h, y: NULL or matrices of dtype.  h may be x or residual itself (same stride).
 *   y8: NULL or the checkpoint of y, taken before y is rounded to dtype: the input that the
 *       following products save for their weight gradients.
 *   h8: NULL or the checkpoint of the rounded h: what zs_rmsnorm_backward can read instead
 *       of h.
 *   rstd: NULL or rows fp32.
 * cols is 1 .. 16384.
 * Errors: ZS_EINVAL on NULL x or weight, no output at all, h and y or y8 and h8 in one place, h
 * in place at another stride, a bad dtype, size, stride, alignment or code, or an eps that is
 * no normal fp32 number above 0. */
zs_status zs_rmsnorm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                     const void* weight, zs_dtype dtype, int64_t rows, int64_t cols, double eps, void* h,
                     int64_t h_stride, void* y, int64_t y_stride, const zs_act* y8, const zs_act* h8, float* rstd,
                     void* stream);

/* Bytes of zs_rmsnorm_backward's workspace (at least 16).  Host only.
 * Errors: ZS_EINVAL on a NULL output, rows < 0 or cols outside 1 .. 16384. */
zs_status zs_rmsnorm_workspace(int64_t rows, int64_t cols, int64_t* bytes);

/* Backward pass of zs_rmsnorm.  With xh = h * rstd and g = dy * weight, in fp32:
 *   dx = rstd * (g - xh * mean(g * xh)) + dh       (the gradient of x and of the residual)
 *   dweight = base + sum over rows of dy * xh
 *   dy: gradient of y; dh: NULL or the gradient that reaches h by other ways.
 *   h or h8: exactly one of them: the saved h, or its checkpoint.
 *   rstd: as zs_rmsnorm wrote it.
 *   dx: rounded once to dtype; may be dy or dh itself (same stride).
 *   dweight: NULL or cols elements of dweight_dtype (bf16, fp16 or fp32): a tensor's place in
 *       a gradient buffer, for instance.  base: NULL or cols elements of the same dtype;
 *       dweight itself adds to what is there.  The sum is rounded once.
 *   workspace: device memory of at least zs_rmsnorm_workspace bytes, 16-byte aligned; may be NULL
 *       when dweight is.
 * Errors: ZS_EINVAL on NULL dy, weight, rstd or dx, neither or both of h and h8, dx in place at
 * another stride, a base without dweight, a missing, small or misaligned workspace, or as zs_rmsnorm. */
zs_status zs_rmsnorm_backward(const void* dy, int64_t dy_stride, const void* dh, int64_t dh_stride, const void* h,
                              int64_t h_stride, const zs_act* h8, const void* weight, const float* rstd,
                              zs_dtype dtype, int64_t rows, int64_t cols, void* dx, int64_t dx_stride, void* dweight,
                              zs_dtype dweight_dtype, const void* base, void* workspace, int64_t workspace_bytes,
                              void* stream);

/* Bytes of zs_act_wgrad's workspace (at least 16).  Host only.
 * Errors: ZS_EINVAL on a NULL output, rows < 0, cols < 1, outs < 1 or sizes past one launch. */
zs_status zs_act_wgrad_workspace(int64_t rows, int64_t cols, int64_t outs, int64_t* bytes);

/* Weight gradient of a linear layer y = x W^T from the checkpoint of its input:
 *   dw[n][k] = base[n][k] + sum over tokens t of dy[t][n] * x8[t][k]
 * on the matrix cores: x8's values take part in dy's dtype (for bf16 as they are, but that
 * those below its normal numbers may count as zero; for fp16 see above), products are exact
 * and summed in fp32, the result is rounded once to dw_dtype.
 *   x8: checkpoint of rows x cols;  dy: rows x outs, bf16 or fp16.
 *   dw: outs x cols of dw_dtype (dy's dtype or fp32), or cols x outs when in_major is not 0
 *       (weights kept as (in, out)); a view of the flat gradient buffer, for instance.
 *   base: NULL or a matrix of dw's dtype, shape and stride; dw itself adds to what is there
 *       (gradient accumulation).
 *   workspace: device memory of at least zs_act_wgrad_workspace bytes, 16-byte aligned.
 * Errors: ZS_EINVAL on a NULL pointer, bad dtype, code, size, stride or alignment, or a missing
 * or small workspace; ZS_EUNSUPPORTED for a dw_dtype that is neither dy's nor fp32. */
zs_status zs_act_wgrad(const zs_act* x8, int64_t rows, int64_t cols, const void* dy, zs_dtype dy_dtype,
                       int64_t dy_stride, int64_t outs, void* dw, zs_dtype dw_dtype, int64_t dw_stride,
                       int32_t in_major, const void* base, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_ACT_H */

/*
 * iq_fp4.h -- C-ABI of libiqcodec.so, third part: weights of 4 bits on AMD
 * Instinct MI355X (gfx950).
 *   - rows as 4-bit floats with a power of two for each 32 values, and back;
 *   - products of activations with such a weight, dense or with a weight per
 *     expert, without a gradient: operators of serving.
 *
 * The conventions are those of iq_layers.h.
 */
#ifndef IQ_FP4_H
#define IQ_FP4_H

#include "iq_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values that share a scale. */
enum { IQ_GROUP = 32 };

/* Rows as 4-bit floats in groups of 32 values that share a power of two (the
 * MXFP4 format of the OCP microscaling specification, codes and scales apart):
 *   scale byte s stands for 2^(s - 127), 255 for NaN;      [rows][cols/32]
 *   a code, sign bit first, for +-(0, 1/2, 1, 3/2, 2, 3, 4, 6); byte i of a row
 *   has the codes of values 2i (low bits) and 2i + 1.      [rows][cols/2]
 * Of a group with the largest magnitude m, 2^(s - 127) = 2^(floor(log2 m) - 2),
 * not below 2^-127, and a code is the nearest to x / 2^(s - 127), halves to the
 * even code, 6 beyond 6, with the sign of x.  A group of zeros has s = 0.  A group
 * that holds a NaN or an infinity is reported as IQ_ERR_NONFINITE and written as
 * zeros.  cols is a multiple of 32; ldc and lds are the strides of rows in bytes. */
iq_status_t iq_quantize_groups(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t rows,
                               int64_t cols, uint8_t* codes, int64_t ldc, uint8_t* scale,
                               int64_t lds, int32_t* status, hipStream_t stream);

/* What they stand for, rounded once to the type of y (exact in fp32 and bf16 up to
 * their largest value). */
iq_status_t iq_dequantize_groups(const uint8_t* codes, int64_t ldc, const uint8_t* scale,
                                 int64_t lds, int64_t rows, int64_t cols, iq_dtype_t out_dtype,
                                 void* y, int64_t ldy, hipStream_t stream);

/* y[t][n] = sum_k x[t][k] * w[n][k] with w in that format, [channels][depth], depth
 * a multiple of 32.  Products are exact (fp32 activations below 2^-110 lose what they
 * have below 2^-133, and those below that count as 0), sums in fp32, rounded once to the
 * type of y, which is that of x.
 * NaN and infinities pass as in any product of floats; a value of w beyond fp32 (scale
 * bytes from 253 on) counts as infinite.
 * `workspace`: iq_fp4_linear_workspace(...) bytes, 16-byte aligned (NULL where that
 * is 0); of x only its alignment counts there. */
int64_t iq_fp4_linear_workspace(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t tokens,
                                int64_t channels, int64_t depth);
iq_status_t iq_fp4_linear(iq_dtype_t dtype, const void* x, int64_t ldx, const uint8_t* w,
                          int64_t ldw, const uint8_t* w_scale, int64_t lds, int64_t tokens,
                          int64_t channels, int64_t depth, void* y, int64_t ldy, void* workspace,
                          int64_t workspace_bytes, hipStream_t stream);

/* The same with a weight per expert, w + e * w_stride and w_scale + e * s_stride
 * (bytes), on the rows that iq_int8_expert_matmul describes. */
int64_t iq_fp4_expert_linear_workspace(iq_dtype_t dtype, const void* x, int64_t ldx,
                                       int64_t tokens, int32_t experts, int64_t rows,
                                       int64_t channels, int64_t depth);
iq_status_t iq_fp4_expert_linear(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t tokens,
                                 const int32_t* order, int32_t top_k, const int32_t* offsets,
                                 int32_t experts, int64_t rows, const uint8_t* w, int64_t ldw,
                                 int64_t w_stride, const uint8_t* w_scale, int64_t lds,
                                 int64_t s_stride, int64_t channels, int64_t depth, void* y,
                                 int64_t ldy, void* workspace, int64_t workspace_bytes,
                                 hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IQ_FP4_H */

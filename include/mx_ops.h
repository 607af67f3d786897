/*
 * mx_ops.h - C ABI of the norm between layers and of microscaled operands: a
 * root-mean-square norm with the residual's addition and its gradients, the
 * quantisation of a matrix into blocks of 32 values that share a power-of-two
 * scale, and the linear layer on two matrices held so.
 *
 * Conventions for every entry point: those of layer_ops.h (16-bit matrices are
 * row-major with a row stride that is a multiple of 8 and an address that is a
 * multiple of 16 bytes; sums in fp32; outputs rounded once; asynchronous on
 * `stream`; arguments checked on the host before any CUDA call; argument
 * structures hold 8-byte fields only).
 *
 * A microscaled matrix [rows, cols] is two arrays (the OCP microscaling formats
 * MXFP8 and MXFP4):
 *   data   rows of ceil(cols / 32) blocks, a block's 32 values side by side: e4m3
 *          one byte a value, e2m1 half a byte, the lower half first.  The last
 *          block is filled up with zeros.  Rows lie `ld` BYTES apart, a multiple
 *          of 16; the address is a multiple of 16.
 *   scale  a block's scale is 2^(byte - 127), and byte 255 makes its values NaN.
 *          The bytes lie in tiles of 128 rows by 4 blocks, 512 bytes each, without
 *          gaps: tile (row / 128, block / 4) of ceil(rows / 128) x
 *          ceil(cols / 128), row-major; within it (row % 32) * 16 +
 *          (row / 32 % 4) * 4 + block % 4.  The address is a multiple of 16.  Of a
 *          row that exists the entries behind the last block are 0; entries of
 *          rows that do not exist hold anything.
 */
#ifndef TCGEMM_MX_OPS_H
#define TCGEMM_MX_OPS_H

#include "layer_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MX_E4M3 = 0, /* 8 bits: up to 448, spacing 1/8 of the power of two below */
    MX_E2M1 = 1  /* 4 bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6 */
} mx_format;

/*
 * x [rows, cols] (fp16 or bf16) into microscaled blocks along its rows; with transpose
 * along its columns: the result is then [cols, rows].
 *
 * A block's scale is 2^(floor(log2 amax) - emax), amax its largest magnitude and emax
 * the exponent of the format's largest value (8 of e4m3, 2 of e2m1), at least 2^-127.
 * Its values are divided by that (exactly) and rounded to nearest even; what lies
 * beyond the format's largest value becomes that value.  A block that holds an
 * infinity or a NaN gets scale byte 255.
 */
typedef struct {
    const void *x;
    void *data, *scale;
    long long ldx, ldd;
    long long rows, cols;
    long long dtype, format, transpose;
} mx_quantize_args;
int mx_quantize(const mx_quantize_args *args, gemm_stream_t stream);

/* The values of a microscaled matrix [rows, cols] in fp16 or bf16, rounded to nearest
 * even (what mx_quantize made of such a matrix comes back exactly). */
typedef struct {
    const void *data, *scale;
    void *x;
    long long ldd, ldx;
    long long rows, cols;
    long long dtype, format;
} mx_dequantize_args;
int mx_dequantize(const mx_dequantize_args *args, gemm_stream_t stream);

/*
 * y = act(x w^T + bias) + residual
 *
 *   x         [tokens, k] and w [n, k], microscaled, of one format
 *   bias      [n] of y's type, or NULL
 *   residual  [tokens, n] of y's type, or NULL; may be y itself (same ld)
 *   y         [tokens, n], fp16 or bf16 (dtype)
 */
typedef struct {
    const void *x, *x_scale, *w, *w_scale, *bias, *residual;
    void *y;
    long long ldx, ldw, ldr, ldy;
    long long tokens, k, n;
    long long dtype, act, format;
} mx_linear_args;
int mx_linear(const mx_linear_args *args, gemm_stream_t stream);

/*
 * h = x + residual (rounded to their type), or x where there is no residual;
 * y = h rstd weight with rstd = 1 / sqrt(mean of h^2 over a row + eps)
 *
 *   x, residual  [tokens, dim]; residual may be NULL
 *   weight       [dim] of x's type, 16-byte aligned
 *   h            [tokens, dim], wanted exactly where there is a residual; may be x or
 *                the residual itself (same ld)
 *   y            [tokens, dim] of x's type, or NULL
 *   data, scale  y as a microscaled matrix of `format` (rounded once, from fp32), or
 *                both NULL.  At least one of y and data is wanted
 *   rstd         [tokens] fp32, or NULL
 * The norm is that of h as it is stored.  Squares are summed in fp32: beyond 3e38 a
 * sum is infinite and its row 0.
 */
typedef struct {
    const void *x, *residual, *weight;
    void *h, *y, *data, *scale;
    float *rstd;
    long long ldx, ldr, ldh, ldy, ldd;
    long long tokens, dim;
    long long dtype, format;
    double eps;
} rms_norm_args;
int rms_norm_forward(const rms_norm_args *args, gemm_stream_t stream);

/*
 * Gradients of rms_norm_forward, dy that of y and dh (or NULL) that which reaches h by
 * another way, the residual stream:
 *   dx      = rstd dy weight - h rstd^3 mean(dy weight h) + dh    (of x and of residual)
 *   dweight = sum over tokens of dy h rstd
 *
 *   dy, h, dh, dx [tokens, dim]; dx may be dy or dh itself (same ld)
 *   weight        [dim], 16-byte aligned;  rstd [tokens] fp32, as the forward pass gave it
 *   dx, dweight   each NULL when not wanted
 */
typedef struct {
    const void *dy, *h, *weight, *dh;
    const float *rstd;
    void *dx, *dweight;
    long long lddy, ldh, lddh, lddx;
    long long tokens, dim;
    long long dtype;
    void *workspace;
    long long workspace_bytes;
} rms_norm_grad_args;
int rms_norm_backward(const rms_norm_grad_args *args, gemm_stream_t stream);
int rms_norm_backward_workspace(const rms_norm_grad_args *args, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* TCGEMM_MX_OPS_H */

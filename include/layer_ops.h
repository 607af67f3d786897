/*
 * layer_ops.h - C ABI of the layer operators built on the GEMM's machinery: a
 * linear layer with bias, activation and residual in its epilogue, the gated
 * feed-forward block, and the cross entropy of a vocabulary projection, each
 * with its backward pass; and the clipping of gradients by their global norm.
 *
 * Conventions for every entry point, beside those of gemm_f16.h (status codes,
 * device pointers owned by the caller, asynchronous on `stream`, host-side
 * argument checks before any CUDA call, callable from several host threads):
 *   - Operands are fp16 or bf16 (one type per call), products are accumulated
 *     in fp32 and each output is rounded once, to nearest even.  What one
 *     product of a call hands the next is rounded to that type too: hidden,
 *     dpre, dgate and dup, and d of the loss.  In fp16 they have its range: a
 *     hidden above 65504 is infinite, also when nothing is kept, and of dpre,
 *     dgate and dup nothing is left below 2^-25, so gradients want a loss scale
 *     there.  (d is scaled by the call itself.)
 *   - A matrix is row-major with a row stride ("ld", in elements) of at least
 *     its width.  TMA wants a row stride that is a multiple of 8 and a base
 *     address that is a multiple of 16 bytes, else GEMM_ERR_ALIGN; widths and
 *     heights are free.
 *   - Sizes are 64-bit in the arguments; each must stay below 2^31 - 1024
 *     (GEMM_ERR_DIM), products of sizes need not.  `tokens` may be 0: outputs
 *     with a row per token are then empty, weight gradients zero.
 *   - Outputs may not overlap inputs or each other (GEMM_ERR_ALIAS), except
 *     where an entry says so.  Matrices that interleave without sharing an
 *     element are told apart where their row strides are the same (column
 *     ranges of one buffer); with different strides they are refused.
 *   - Scratch memory comes from the caller as `workspace` (256-byte aligned,
 *     no initial contents needed, free again when the stream has passed the
 *     call).  Its size comes from the *_workspace entry, host-only.
 *   - Every argument structure holds 8-byte fields only; zero it before use.
 */
#ifndef TCGEMM_LAYER_OPS_H
#define TCGEMM_LAYER_OPS_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { LAYER_F16 = 0, LAYER_BF16 = 1, LAYER_F32 = 2 /* grad_clip only */ } layer_dtype;

typedef enum {
    LAYER_ACT_NONE = 0,
    LAYER_ACT_RELU = 1,
    LAYER_ACT_SILU = 2,      /* x / (1 + exp(-x)) */
    LAYER_ACT_GELU = 3,      /* x/2 (1 + erf(x / sqrt 2)) */
    LAYER_ACT_GELU_TANH = 4  /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
} layer_act;

typedef enum { LAYER_LOSS_NONE = 0, LAYER_LOSS_MEAN = 1, LAYER_LOSS_SUM = 2 } layer_reduction;

/*
 * y = act(x w + bias) + residual
 *
 *   x         [tokens, k]       w   [k, n]
 *   bias      [n] of the operands' type, or NULL
 *   residual  [tokens, n], or NULL; may be y itself (same ld)
 *   y         [tokens, n]
 *   preact    [tokens, n], or NULL: receives x w + bias, which linear_backward reads
 */
typedef struct {
    const void *x, *w, *bias, *residual;
    void *y, *preact;
    long long ldx, ldw, ldr, ldy, ldp;
    long long tokens, k, n;
    long long dtype, act;
} linear_args;
int linear_forward(const linear_args *args, gemm_stream_t stream);

/*
 * Gradients of linear_forward: dpre = dy act'(preact), dx = dpre w^T,
 * dw = x^T dpre, dbias = column sums of dpre.  (The residual's is dy itself.)
 *
 *   dy      [tokens, n]      preact  [tokens, n]; may be NULL when act is none
 *   dx      [tokens, k], dw [k, n], dbias [n]; each NULL when not wanted
 */
typedef struct {
    const void *dy, *x, *w, *preact;
    void *dx, *dw, *dbias;
    long long lddy, ldx, ldw, ldp, lddx, lddw;
    long long tokens, k, n;
    long long dtype, act;
    void *workspace;
    long long workspace_bytes;
} linear_grad_args;
int linear_backward(const linear_grad_args *args, gemm_stream_t stream);
int linear_backward_workspace(const linear_grad_args *args, size_t *bytes);

/*
 * The gated feed-forward block:
 *   hidden = act(x w_gate) * (x w_up)       one kernel
 *   y      = hidden w_down + residual       one kernel
 *
 *   x [tokens, dim], w_gate and w_up [dim, ffn], w_down [ffn, dim_out]
 *   residual  [tokens, dim_out], or NULL; may be y itself (same ld)
 *   hidden    [tokens, ffn], always written (the second product reads it)
 *   gate, up  [tokens, ffn]: x w_gate and x w_up for the backward pass, or both NULL
 */
typedef struct {
    const void *x, *w_gate, *w_up, *w_down, *residual;
    void *y, *hidden, *gate, *up;
    long long ldx, ldw_gate, ldw_up, ldw_down, ldr, ldy, ld_hidden, ld_gate, ld_up;
    long long tokens, dim, ffn, dim_out;
    long long dtype, act;
} gated_args;
int gated_ffn_forward(const gated_args *args, gemm_stream_t stream);

/*
 * Gradients of gated_ffn_forward from what it kept:
 *   dhidden = dy w_down^T, dgate = dhidden up act'(gate), dup = dhidden act(gate)
 *   dx = dgate w_gate^T + dup w_up^T, dw_gate = x^T dgate, dw_up = x^T dup, dw_down = hidden^T dy
 *
 * dx, dw_gate and dw_up (together), dw_down: each NULL when not wanted.
 */
typedef struct {
    const void *dy, *x, *w_gate, *w_up, *w_down, *gate, *up, *hidden;
    void *dx, *dw_gate, *dw_up, *dw_down;
    long long lddy, ldx, ldw_gate, ldw_up, ldw_down, ld_gate, ld_up, ld_hidden;
    long long lddx, lddw_gate, lddw_up, lddw_down;
    long long tokens, dim, ffn, dim_out;
    long long dtype, act;
    void *workspace;
    long long workspace_bytes;
} gated_grad_args;
int gated_ffn_backward(const gated_grad_args *args, gemm_stream_t stream);
int gated_ffn_backward_workspace(const gated_grad_args *args, size_t *bytes);

/*
 * Cross entropy of h w^T against target, without the logits in memory:
 *   lse[t]  = ln sum_v exp(h_t . w_v)
 *   loss[t] = lse[t] - h_t . w_target[t], 0 where target[t] == ignore_index
 *
 *   h [tokens, dim], w [vocab, dim] (a row per word), target [tokens] int64
 *   lse   [tokens] fp32
 *   loss  fp32: [tokens] (none), or one value: the sum of the losses (sum), or that
 *         over the number of targets that count (mean; 0 when none counts)
 * A target outside [0, vocab) that is not ignore_index makes its loss NaN.
 */
typedef struct {
    const void *h, *w;
    const long long *target;
    float *loss, *lse;
    long long ldh, ldw;
    long long tokens, dim, vocab;
    long long dtype, ignore_index, reduction;
    void *workspace;
    long long workspace_bytes;
} loss_args;
int linear_cross_entropy(const loss_args *args, gemm_stream_t stream);
int linear_cross_entropy_workspace(const loss_args *args, size_t *bytes);

/*
 * Its gradients: d[t][v] = (exp(h_t . w_v - lse[t]) - [v = target[t]]) weight[t],
 * dh = d w, dw = d^T h, with weight[t] = grad_loss[t] (none), grad_loss[0] (sum) or
 * grad_loss[0] / targets that count (mean), and 0 for an ignored row.
 *
 * The logits are computed again, a piece of the vocabulary at a time: d of one
 * piece is held in 16 bits in the workspace, relative to the largest |weight|; for
 * dh in fp16 with reduction none relative to each row's own, in a second copy.
 * Any workspace from the _workspace
 * entry's size for piece = 256 on will do; *piece (a multiple of 256) asks for
 * the size of that piece, or all of vocab when smaller.  More than one piece
 * also takes tokens x dim fp32 for dh's running sum.
 *
 *   dh [tokens, dim], dw [vocab, dim]
 */
typedef struct {
    const void *h, *w;
    const long long *target;
    const float *lse, *grad_loss;
    void *dh, *dw;
    long long ldh, ldw, lddh, lddw;
    long long tokens, dim, vocab;
    long long dtype, ignore_index, reduction;
    void *workspace;
    long long workspace_bytes;
} loss_grad_args;
int linear_cross_entropy_backward(const loss_grad_args *args, gemm_stream_t stream);
int linear_cross_entropy_backward_workspace(const loss_grad_args *args, long long piece, size_t *bytes);

/*
 * norm = sqrt(sum of squares of every entry of every tensor);
 * dst[i] = src[i] * min(1, max_norm / (norm + eps)).
 *
 *   tensors   how many; src, dst, count, dtype are HOST arrays of that length, read
 *             during the call only
 *   src, dst  dense device arrays of count[i] entries of dtype[i] (fp16, bf16 or
 *             fp32), aligned to their type; dst[i] may be src[i] (in place).
 *             Different tensors may not overlap (not checked)
 *   norm      one fp32 on the device, or NULL
 * An infinite norm scales by 0 and a NaN norm by NaN, as the formula says.  Squares
 * are summed in fp32: a norm above 1e19 comes out infinite, entries below 1e-23 count
 * as 0.
 */
typedef struct {
    const void *const *src;
    void *const *dst;
    const long long *count;
    const int *dtype;
    float *norm;
    void *workspace;
    long long tensors;
    double max_norm, eps;
    long long workspace_bytes;
} grad_clip_args;
int grad_clip(const grad_clip_args *args, gemm_stream_t stream);
int grad_clip_workspace(long long tensors, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* TCGEMM_LAYER_OPS_H */

/*
 * zero_layer.h -- the layer operators of libzero (AMD Instinct MI355X, gfx950):
 * what runs between the fetch of a layer's tensors and the optimizer step of
 * zero.h, whose conventions hold here too (statuses, synchronous argument checks,
 * error text, caller-owned device memory, caller's stream).
 */
#ifndef ZERO_LAYER_H
#define ZERO_LAYER_H

#include "zero.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * What runs between zero_gather_tensors and the optimizer step for a linear
 * layer: the product with the fetched weights, its gradient by the layer's input,
 * and its gradient by the weights, written or accumulated in place into the flat
 * gradient buffer whose slices are the step's replicas ("ZeRO Optimizer", "ZeRO
 * Stages": stage 3 gathers the parameters before each forward and backward pass;
 * "Performance Optimization", gradient accumulation; the contiguous gradient
 * buffer of "Why does not the stage 3 implementation use broadcast and
 * reduce-scatter?"), and dropout, whose mask is recomputed wherever it is needed.
 * The pages name these passes and give no formulas; those are:
 *
 *   forward            z  = x W^T + b,   y = residual + D(act(z))
 *   gradient by input  dx = D'(dz W) * act'(z)        (z, D of the layer below,
 *                                                      whose output x was)
 *   gradient by weight dW = [dW +] dz^T x,  db = [db +] sum of dz over its rows
 *   dropout            y  = residual + D(x)
 *   its gradient       dz = D'(dy) * act'(z)
 *
 * with M rows (tokens), K inputs and N outputs. Operands are bf16, sums fp32, and
 * every result is rounded once, from fp32, when it is stored; z is rounded to bf16
 * where it is stored, and the forward's act takes it unrounded.
 *
 * Matrices are row-major with a row length ("ld", in elements) of at least their
 * columns, which need not be a multiple of anything; the elements between a row's
 * columns and its ld are never written and never take part. Pointers need the
 * alignment of their element only. Rows of a length that is a multiple of 8 from
 * a 16-byte aligned base take the faster path; its 16-byte loads may read, and
 * ignore, up to 7 elements behind a row's last column inside that column's
 * 16-byte unit. A matrix with no elements may be NULL. All calls enqueue on
 * `stream` and may be captured; nothing is kept between calls, so the workspace is
 * free for other use on the same stream once a call's kernels are enqueued, but
 * calls that may run at the same time (two streams, two captured graphs) need
 * workspaces of their own.
 * Results do not depend on timing: the splits of a long sum are joined in order.
 * Outputs must not overlap inputs or each other, with one exception: an output may
 * be exactly an elementwise input (same address, type and ld): y over residual, dx
 * over preact, dz over dy or preact, y over x in zero_dropout_add.
 */

/* How a weight lies in memory: [N, K] (a row per output) or [K, N]. */
typedef enum { ZERO_W_OUT_IN = 0, ZERO_W_IN_OUT = 1 } zero_weight_layout;

/*
 * GELU is the tanh form, z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))); SiLU is
 * z / (1 + exp(-z)). ReLU's slope is 1 where z > 0 and 0 elsewhere, at a NaN too
 * (whose ReLU is NaN); the other slopes at a NaN are NaN.
 */
typedef enum {
    ZERO_ACT_NONE = 0,
    ZERO_ACT_RELU = 1,
    ZERO_ACT_GELU = 2,
    ZERO_ACT_SILU = 3
} zero_activation;

/*
 * Dropout of an [M, N] matrix. Element (i, j) is dropped when its draw is below
 * thr = p * 65536, rounded to nearest even; kept elements are multiplied by
 * 65536 / (65536 - thr), dropped ones are 0 whatever they held. The draw is 16
 * bits of Philox4x32-10 (Salmon et al. 2011) with key (seed low, seed high) and
 * counter (j / 8, i, offset low, offset high): word (j % 8) / 2, its low half for
 * even j. No mask is stored: the backward pass passes the same seed and offset.
 * counter_dev, if not NULL, is a device int64 that is added to offset when the
 * kernel runs, so that a captured call draws anew once its program has advanced
 * it. p = 0 (in a zeroed struct) is no dropout.
 * Errors of every call that takes one: ZERO_E_INVAL (p not in [0, 1 - 2^-16], or
 * NaN), ZERO_E_ALIGN (counter_dev not 8-byte aligned).
 */
typedef struct {
    double p;
    uint64_t seed;
    uint64_t offset;
    const int64_t* counter_dev;
} zero_dropout;

/*
 * Which product a workspace is for, and its size. The largest of a program's
 * calls serves all of them on one stream. 0 if none is needed (workspace_dev may
 * then be NULL); arguments out of range give 0. It holds for operands at any
 * alignment; products of at most 16 rows that run in one launch take NULL too.
 */
typedef enum {
    ZERO_LINEAR_FORWARD = 0,
    ZERO_LINEAR_GRAD_INPUT = 1,
    ZERO_LINEAR_GRAD_WEIGHT = 2
} zero_linear_kind;

size_t zero_linear_workspace_bytes(int32_t kind, int32_t w_layout, int64_t M, int64_t K, int64_t N);

/*
 * y = residual + D(act(x W^T + bias)), and, if preact is given, preact = x W^T +
 * bias in bf16 (what the gradients of the activation need).
 */
typedef struct {
    int64_t M, K, N;
    const uint16_t* x;             /* bf16 [M, K] */
    int64_t ld_x;
    const uint16_t* w;             /* bf16, as w_layout says */
    int64_t ld_w;
    int32_t w_layout;              /* zero_weight_layout */
    int32_t act;                   /* zero_activation */
    const uint16_t* bias;          /* bf16 [N], may be NULL */
    const void* residual;          /* [M, N] of y's type, may be NULL */
    int64_t ld_residual;
    void* y;                       /* [M, N] */
    int64_t ld_y;
    int32_t y_dtype;               /* ZERO_BF16 or ZERO_F32 */
    int32_t reserved;
    uint16_t* preact;              /* bf16 [M, N], may be NULL */
    int64_t ld_preact;
    zero_dropout dropout;
    void* workspace_dev;
    size_t ws_bytes;
} zero_linear_args;

/*
 * Errors of the three products: ZERO_E_INVAL (NULL args or matrix, an unknown
 * layout, activation or type, a dropout out of domain, an activation's gradient
 * without preact, overlap), ZERO_E_ALIGN (a pointer not aligned to its element, a
 * workspace not to 16 bytes), ZERO_E_RANGE (a size outside [0, 2^31 - 1], an output
 * of more than 2^29 rows or columns or 2^23 tiles of 128 x 128, an ld below its
 * columns or above 2^40, a workspace below zero_linear_workspace_bytes where the call
 * needs one), ZERO_E_HIP.
 */
int zero_linear_forward(const zero_linear_args* args, void* stream);

/*
 * dx = D'(dz W) * act'(preact): the gradient by a linear layer's input, taken on
 * through the dropout and activation of the layer below if they are given (the
 * dropout of an [M, K] matrix). act NONE: preact is not read and may be NULL.
 */
typedef struct {
    int64_t M, K, N;
    const uint16_t* dz;            /* bf16 [M, N] */
    int64_t ld_dz;
    const uint16_t* w;             /* bf16, as w_layout says */
    int64_t ld_w;
    int32_t w_layout;
    int32_t act;
    const uint16_t* preact;        /* bf16 [M, K] */
    int64_t ld_preact;
    void* dx;                      /* [M, K] */
    int64_t ld_dx;
    int32_t dx_dtype;              /* ZERO_BF16 or ZERO_F32 */
    int32_t reserved;
    zero_dropout dropout;
    void* workspace_dev;
    size_t ws_bytes;
} zero_linear_grad_input_args;

int zero_linear_grad_input(const zero_linear_grad_input_args* args, void* stream);

/*
 * dW = dz^T x and, if dbias is given, dbias = the sum of dz over its rows, in the
 * weight's own layout and the type of the gradient replicas; accumulate != 0 adds
 * to what dw and dbias hold (one rounding, of the sum). With M = 0 they become 0,
 * or stay.
 */
typedef struct {
    int64_t M, K, N;
    const uint16_t* dz;            /* bf16 [M, N] */
    int64_t ld_dz;
    const uint16_t* x;             /* bf16 [M, K] */
    int64_t ld_x;
    void* dw;                      /* [N, K] or [K, N] */
    int64_t ld_dw;
    void* dbias;                   /* [N], may be NULL */
    int32_t w_layout;
    int32_t grad_dtype;            /* ZERO_BF16 or ZERO_F32, of dw and dbias */
    int32_t accumulate;
    int32_t reserved;
    void* workspace_dev;
    size_t ws_bytes;
} zero_linear_grad_weight_args;

int zero_linear_grad_weight(const zero_linear_grad_weight_args* args, void* stream);

/*
 * y = residual + D(x), and dz = D'(dy) * act'(preact), over [M, N]. x and dy are
 * in x_dtype, y and dz (and the residual) in y_dtype, each ZERO_BF16 or ZERO_F32;
 * preact is bf16. Errors as for the products; zero_dropout_add takes no act or
 * preact, zero_dropout_grad no residual (ZERO_E_INVAL).
 */
typedef struct {
    int64_t M, N;
    const void* x;                 /* x, or dy */
    int64_t ld_x;
    const void* residual;          /* may be NULL */
    int64_t ld_residual;
    const uint16_t* preact;        /* bf16; not read if act is NONE */
    int64_t ld_preact;
    void* y;                       /* y, or dz */
    int64_t ld_y;
    int32_t x_dtype;
    int32_t y_dtype;
    int32_t act;
    int32_t reserved;
    zero_dropout dropout;
} zero_dropout_args;

int zero_dropout_add(const zero_dropout_args* args, void* stream);
int zero_dropout_grad(const zero_dropout_args* args, void* stream);

/*
 * The norm of a block's rows and its gradient ("ZeRO Stages": the norms' weights are
 * among the tensors that stage 3 gathers and whose gradients the step averages; the
 * pages give no formulas). Over a row x of N columns, with w and b of the norm:
 *
 *   forward    s = residual + x                              (or s = x, nothing stored)
 *              mean = sum(s) / N,  rstd = 1 / sqrt(sum((s - mean)^2) / N + eps)
 *              y = (s - mean) rstd w + b
 *   gradient   h = (s - mean) rstd,  g = dy w
 *              dx = residual_grad + rstd (g - sum(g) / N - h sum(g h) / N)
 *              dw = [dw +] sum over rows of dy h,  db = [db +] sum over rows of dy
 *
 * ZERO_NORM_RMS takes mean as 0 and leaves out sum(g) / N. s is rounded to its own type
 * before it is normed: the backward pass reads what the forward pass normed, and a call
 * with a residual gives what an addition and a call without one give. Sums and
 * statistics are fp32, the variance from the differences to the mean, and y from the mean
 * before it is rounded to its place in stats (the gradient's h has that one: it is off by
 * 2^-25 mean / sigma). A row of one value gives y = b, and with eps 0 rstd = inf and, by the
 * formula, NaN. A NaN in a row makes that row's y NaN, an infinity too, except that in an
 * RMS norm, whose rstd is then 0, it does so in its own place and leaves b in the others; so
 * does (without the NaN) a row whose squares pass fp32.
 */
typedef enum { ZERO_NORM_LAYER = 0, ZERO_NORM_RMS = 1 } zero_norm_kind;

/*
 * y, sum and stats of the rows of x. sum is required with a residual and must be NULL
 * without one. y or sum may be exactly x or residual (same address, type and ld), not
 * each other. One launch, no workspace.
 */
typedef struct {
    int64_t M, N;
    const void* x;                 /* [M, N] of x_dtype */
    int64_t ld_x;
    const void* residual;          /* [M, N] of sum_dtype, may be NULL */
    int64_t ld_residual;
    const uint16_t* weight;        /* bf16 [N], may be NULL: ones */
    const uint16_t* bias;          /* bf16 [N], may be NULL: zeros */
    void* y;                       /* [M, N] of y_dtype */
    int64_t ld_y;
    void* sum;                     /* [M, N] of sum_dtype: s */
    int64_t ld_sum;
    float* stats;                  /* [M, 2]: mean and rstd of each row, may be NULL */
    int32_t x_dtype;               /* ZERO_BF16 or ZERO_F32, each of the three */
    int32_t sum_dtype;
    int32_t y_dtype;
    int32_t kind;                  /* zero_norm_kind */
    double eps;
} zero_norm_args;

/*
 * Errors of both calls: ZERO_E_INVAL (NULL args or matrix, an unknown kind or type, eps
 * outside [0, 1e30] or NaN, a residual without sum or a sum without residual, overlap),
 * ZERO_E_ALIGN (a pointer not aligned to its element, a workspace not to 16 bytes),
 * ZERO_E_RANGE (M outside [0, 2^31 - 1], N outside [0, 2^24], an ld below its columns or
 * above 2^40, a workspace below zero_norm_workspace_bytes), ZERO_E_HIP.
 */
int zero_norm_forward(const zero_norm_args* args, void* stream);

/*
 * The gradient by the rows, with what the residual stream's own gradient adds, and the
 * gradients by weight and bias, reduced over the rows in an order that depends on the
 * sizes alone. stats are the forward pass's. dx may be exactly dy, x or residual_grad.
 * dweight and dbias may each be NULL; without both no workspace is needed. With M = 0
 * they become 0, or stay.
 */
typedef struct {
    int64_t M, N;
    const void* dy;                /* [M, N] of dy_dtype */
    int64_t ld_dy;
    const void* x;                 /* [M, N] of x_dtype: s of the forward pass */
    int64_t ld_x;
    const uint16_t* weight;        /* bf16 [N], may be NULL: ones */
    const float* stats;            /* [M, 2] */
    const void* residual_grad;     /* [M, N] of dx_dtype, may be NULL */
    int64_t ld_residual_grad;
    void* dx;                      /* [M, N] of dx_dtype */
    int64_t ld_dx;
    void* dweight;                 /* [N] of grad_dtype, may be NULL */
    void* dbias;                   /* [N] of grad_dtype, may be NULL */
    int32_t dy_dtype;              /* ZERO_BF16 or ZERO_F32, each of the four */
    int32_t x_dtype;
    int32_t dx_dtype;
    int32_t grad_dtype;
    int32_t kind;                  /* zero_norm_kind */
    int32_t accumulate;
    void* workspace_dev;
    size_t ws_bytes;
} zero_norm_grad_args;

/* Bytes of zero_norm_grad's workspace; 0 for sizes out of range. */
size_t zero_norm_workspace_bytes(int64_t M, int64_t N);

int zero_norm_grad(const zero_norm_grad_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_LAYER_H */

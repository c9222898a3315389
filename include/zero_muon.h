/*
 * zero_muon.h -- the step of a layer's matrices by an orthogonalised momentum, in
 * libzero (AMD Instinct MI355X, gfx950). It stands beside the Adam step of zero.h for
 * the tensors that are matrices; that header's conventions hold here too (statuses,
 * synchronous argument checks, error text, caller-owned device memory, caller's stream).
 */
#ifndef ZERO_MUON_H
#define ZERO_MUON_H

#include "zero.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One rank's step of a shard that holds matrices ("[REQUEST] Direct Correspondence
 * between Gradient and Optimizer States to Reduce Communication", "Problem": the owner
 * of a slice updates it; the pages name Adam and leave other optimizers open). The
 * optimizer is the momentum whose matrices are replaced by their nearest
 * semi-orthogonal ones before the update ("Muon", K. Jordan et al. 2024, published
 * formulas):
 *
 *   momentum        m' = mu m + g,   u = g + mu m'  (nesterov)  or  u = m'
 *   orthogonalise   X = u / (|u| + eps),  |u| the root of the sum of squares
 *                   X <- a X + (b A + c A A) X,  A = X X^T,   `steps` times
 *                   o = scale X
 *   update          p' = p (1 - lr weight_decay) - lr o,   slot = bf16(p')
 *
 * The first and the last go by element, over the shard; the middle one needs whole
 * matrices, so a matrix that shards cut is put together in between (an all-gather of
 * the shards of u). g is zero_reduce_shard's. All calls enqueue on `stream`, may be
 * captured, and keep nothing between calls; pointers need the alignment of their
 * element only.
 */

/*
 * m' and u over n elements, each one fp32 operation per product and sum, u rounded once.
 * mu is rounded once to fp32. stats_dev (may be NULL): where its overflow flag is set
 * when the kernel runs, nothing is written. u may be exactly grad (same type).
 * Errors: ZERO_E_INVAL (NULL, mu outside [0, 1) or NaN, an unknown type, overlap),
 * ZERO_E_ALIGN, ZERO_E_RANGE (n outside [0, 2^40]), ZERO_E_HIP.
 */
typedef struct {
    int64_t n;
    const void* grad;              /* [n] of grad_dtype: averaged, unscaled */
    float* momentum;               /* [n], updated in place */
    void* u;                       /* [n] of u_dtype */
    int32_t grad_dtype;            /* ZERO_BF16 or ZERO_F32, both */
    int32_t u_dtype;
    int32_t nesterov;
    int32_t reserved;
    double mu;
    const zero_stats* stats_dev;
} zero_muon_momentum_args;

int zero_muon_momentum(const zero_muon_momentum_args* args, void* stream);

/*
 * p' and, if slot is given, its bf16 value (nearest, ties to even)
 * over n elements: p * fp32(1 - lr weight_decay) - fp32(lr) * o, one fp32 operation
 * each. stats_dev as above. Errors as above (lr and weight_decay finite, >= 0).
 */
typedef struct {
    int64_t n;
    float* p;                      /* [n], updated in place */
    const uint16_t* o;             /* bf16 [n] */
    uint16_t* slot_bf16;           /* [n], may be NULL */
    double lr, weight_decay;
    const zero_stats* stats_dev;
} zero_muon_update_args;

int zero_muon_update(const zero_muon_update_args* args, void* stream);

/*
 * Orthogonalise `batch` matrices of rows x cols, of any shape. Matrix k lies at
 * x + k * stride_x, its rows ld_x elements apart; o likewise. coefficients: host array
 * of `steps` triples a, b, c, or NULL for (3.4445, -4.7750, 2.0315) in every step.
 *
 * o is bf16. The products run on the matrix cores, each as three of fp16 operands with fp32
 * sums: X, A and b A + c A A are pairs of fp16 numbers, 22 bits and a sign, the diagonals of the
 * last two fp32. A step multiplies by a what roundings leave in directions that x does not
 * hold, whatever number format they were made in. Before o is rounded the result is therefore,
 * with the default coefficients, at most 2^-20 times the product of the steps' a's of its norm
 * from the formula's (5e-4 for five steps; a model of the roundings gives 2e-4 at rank
 * 1, 1e-5 at rank 32 and 1e-6 for normal numbers), 1 to 4 times what fp32 operations leave. Steps whose a's,
 * those below 1 in magnitude left out, multiply to more than 2^13 are refused (with the default
 * coefficients more than seven): a matrix of low rank would come out of them, in 32 bits, wrong
 * in the second digit. X's elements must stay below 16 and those of A and b A + c A A off their
 * diagonals below 64 (with the default coefficients none passes 3); beyond, every element of o that the formula makes of such an element is NaN: all of its matrix,
 * but for the rows (of a matrix taller than wide: columns) that an element of the last step's
 * b A + c A A does not belong to. A matrix of zeros gives zeros. A matrix that holds an infinity
 * or a NaN gives NaN in all its elements, and does not reach the others. The sum of squares
 * is fp64: no scale of x overflows it.
 * Matrices are processed in groups whose intermediate results take 4 GiB at most, one
 * matrix at least. The same call gives the same bits; how sums are split, and so a
 * result's last bits, depends on the sizes and on how many matrices there are.
 * Errors: ZERO_E_INVAL (NULL, an unknown type, steps outside [1, 64], eps not in
 * [1e-30, 1e30], scale or a coefficient not finite or beyond 1e4 in magnitude, a's that multiply
 * to more than 2^13, overlap of the extents of x, o and the workspace), ZERO_E_ALIGN (a pointer not aligned to its element, a workspace
 * not to 16 bytes), ZERO_E_RANGE (batch outside [0, 2^31 - 1], the smaller side above 2^15
 * or the larger above 2^20, an ld below cols or above 2^40, a batch stride below a
 * matrix's extent or above 2^50, a workspace below zero_orthogonalize_workspace_bytes),
 * ZERO_E_HIP.
 */
typedef struct {
    int64_t batch, rows, cols;
    const void* x;
    int64_t ld_x, stride_x;        /* elements; stride_x is not read if batch is 1 */
    uint16_t* o;                   /* bf16 */
    int64_t ld_o, stride_o;
    int32_t x_dtype;               /* ZERO_BF16 or ZERO_F32 */
    int32_t steps;
    const double* coefficients;
    double eps, scale;
    void* workspace_dev;
    size_t ws_bytes;
} zero_orthogonalize_args;

/* Bytes of the workspace, the same for every x, o and steps; 0 for sizes out of range. */
size_t zero_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);

int zero_orthogonalize(const zero_orthogonalize_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_MUON_H */

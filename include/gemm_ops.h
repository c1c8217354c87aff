/*
 * gemm_ops.h -- C ABI of the expert-layer operators of libtcgemm.so: FP8
 * matrices with a scale for each block of 128, their products, the routing of
 * tokens to experts, and the weighted combination of the experts' rows.
 *
 * Conventions are gemm.h's: device pointers owned by the caller, leading
 * dimensions and strides in ELEMENTS, work enqueued on the caller's stream
 * without synchronising, a gemm_status_t returned, gemm_last_error() for the
 * message.  Index arrays live on the device and are int32.
 *
 * Matrices that are only read, row by row (X of the quantisation, logits, Y and
 * grad), may have a row pitch of 0: one row that stands for all of them.
 *
 * Element types: `type` arguments are gemm_out_t for FP32 / BF16 / FP16 data
 * and gemm_dtype_t's GEMM_E4M3 / GEMM_E5M2 for FP8 data.
 */
#ifndef TCGEMM_GEMM_OPS_H
#define TCGEMM_GEMM_OPS_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a matrix is cut into blocks that share a scale. */
typedef enum {
    GEMM_BLOCK_ROW = 0,  /* 1 x 128: 128 neighbouring columns of one row      */
    GEMM_BLOCK_COL = 1,  /* 128 x 1: 128 neighbouring rows of one column      */
    GEMM_BLOCK_TILE = 2  /* 128 x 128                                         */
} gemm_block_t;

/*
 * gemm_quantize_block -- FP8 values and block scales of `batch` matrices X of
 * rows x cols:
 *
 *     scale = max(max |x| over the block / top, 2^-126),
 *     q     = x * (1 / scale) rounded to nearest even,
 *
 * top = 448 (GEMM_E4M3) or 57344 (GEMM_E5M2), so q * scale stands for x.  The
 * blocks at the right and lower edge hold what is there.  An infinity makes
 * its block's scale infinite and a NaN stays one: either way the products
 * that read the block do not come out finite.
 *
 *   type, X      element type (gemm_out_t) and data; row pitch ldx >= cols,
 *                matrices x_stride apart
 *   to, Q        GEMM_E4M3 or GEMM_E5M2 bytes, row pitch ldq >= cols, matrices
 *                q_stride apart
 *   block        gemm_block_t
 *   S            scales: element (i, j) of a matrix's ceil-divided scale array
 *                at S[i * s_row + j * s_col], matrices s_batch apart
 *   slots        NULL, or rows x copies output rows (GEMM_BLOCK_ROW, batch 1):
 *                row r of X goes to rows slots[r * copies .. + copies) of Q
 *                and S, which have out_rows rows; entries outside
 *                [0, out_rows) are skipped, rows no entry names keep what they
 *                hold.  Entries are distinct.
 */
GEMM_API int gemm_quantize_block(int64_t batch, int64_t rows, int64_t cols, int type, const void *X, int64_t ldx,
                                 int64_t x_stride, int block, int to, void *Q, int64_t ldq, int64_t q_stride,
                                 float *S, int64_t s_row, int64_t s_col, int64_t s_batch, const int32_t *slots,
                                 int64_t copies, int64_t out_rows, struct CUstream_st *stream);

/* Block scales of one operand of a product: the scale of K-block kb
 * (128 values of K) for row (of A) or column (of B) i is
 * scale[kb * stride_k + (i / block) * stride_i], block being 1 or 128. */
typedef struct {
    const float *scale;
    int64_t stride_k;
    int64_t stride_i;
    int32_t block;
    int32_t reserved;
} gemm_block_scale_t;

/*
 * gemm_run_scaled -- the product of two FP8 matrices with block scales,
 *
 *   C[m][n] = act(alpha * sum_kb sa(m, kb) * sb(n, kb) *
 *                         sum_{k in kb} A[m][k] * B[k][n] + beta * C + bias[n]).
 *
 * Products within a K-block are exact and summed in FP32 in Tensor Memory; the
 * scaled blocks are summed in FP32 registers, the two scales' product formed
 * first (it must be finite).  The activations keep a NaN (gemm_run_ex's ReLU
 * gives 0 for one).
 *
 *   dtype        GEMM_E4M3 or GEMM_E5M2, both operands
 *   A, lda       a_major 0: row-major, element (m, k) at A[m * lda + k],
 *                lda >= K; 1: at A[k * lda + m], lda >= M
 *   B, ldb       b_major 0: row-major, element (k, n) at B[k * ldb + n],
 *                ldb >= N; 1: at B[n * ldb + k], ldb >= K
 *   a_scale, b_scale  their block scales
 *   C, ldc, epi  as gemm_run_ex (epi NULL: FP32 C, no epilogue)
 * So a layer's Y = X W^T, its dX = dY W and its dW = dY^T X all read their
 * operands as they were stored.  Operands TMA cannot address (base or row
 * pitch not a multiple of 16 bytes) are first copied into a stream-ordered
 * workspace, as in gemm_run.
 */
GEMM_API int gemm_run_scaled(int64_t M, int64_t N, int64_t K, int dtype, const void *A, int64_t lda, int a_major,
                             const gemm_block_scale_t *a_scale, const void *B, int64_t ldb, int b_major,
                             const gemm_block_scale_t *b_scale, void *C, int64_t ldc, const gemm_epilogue_t *epi,
                             struct CUstream_st *stream);

/*
 * gemm_run_experts -- the product of each expert's rows with its own matrix:
 * for e < experts and offsets[e] <= r < offsets[e + 1],
 *
 *   C[r][:] = act(alpha * (A[r][:] . B_e) under the block scales).
 *
 *   rows         rows of A and C (the offsets are clamped to it)
 *   A, lda       row-major FP8, rows in expert order; a_scale one per row
 *                (block 1)
 *   offsets      experts + 1 ascending int32 in device memory; an expert may
 *                have no row; rows of C outside every expert keep what they
 *                hold
 *   B, ldb, b_expert  b_major as gemm_run_scaled, experts b_expert elements
 *                apart; b_scale for expert 0, those of expert e being
 *                b_scale_expert elements further each
 *   epi          alpha, activation and output type; beta 0 and no bias
 * B's base, pitch and b_expert must be multiples of 16 bytes
 * (GEMM_ERR_UNSUPPORTED otherwise: weights are laid out once; an expert of one
 * stored row has no pitch); A is copied into a workspace where it is not.  At
 * most 1024 experts.
 */
GEMM_API int gemm_run_experts(int64_t rows, int64_t N, int64_t K, int64_t experts, int dtype, const void *A,
                              int64_t lda, const gemm_block_scale_t *a_scale, const int32_t *offsets, const void *B,
                              int64_t ldb, int64_t b_expert, int b_major, const gemm_block_scale_t *b_scale,
                              int64_t b_scale_expert, void *C, int64_t ldc, const gemm_epilogue_t *epi,
                              struct CUstream_st *stream);

typedef enum { GEMM_SCORE_SOFTMAX = 0, GEMM_SCORE_SIGMOID = 1 } gemm_score_t;
typedef enum { GEMM_GROUP_MAX = 0, GEMM_GROUP_TOP2 = 1 } gemm_group_score_t;

typedef struct {
    int32_t top_k;        /* experts a token takes, 1 .. 32                    */
    int32_t score;        /* gemm_score_t                                      */
    int32_t groups;       /* experts come in this many equal groups (1: none)  */
    int32_t top_groups;   /* groups a token may choose from, 1 .. groups       */
    int32_t group_score;  /* gemm_group_score_t                                */
    int32_t renormalize;  /* divide a token's weights by their sum             */
    float scale;          /* and multiply them by this                         */
} gemm_route_t;

/*
 * gemm_route -- routes tokens to experts and orders the (token, choice) pairs
 * by expert.
 *
 * Scores s = softmax or sigmoid of a token's logits.  Experts are ranked by
 * key = s + bias (by the logits themselves without a bias: the same order
 * where scores differ); with groups, a group is worth its largest key or the
 * sum of its two largest (scores, without a bias), and only the top_groups
 * best groups take part.  The top_k largest keys are chosen, in descending
 * order; ties go to the lower index.  weight = scale * s, divided by the sum
 * of the token's chosen s when `renormalize` (and that sum is not 0).  A logit
 * of -inf or NaN masks its expert: it has score 0 and is not chosen, nor is an
 * expert whose key is NaN or -inf.  Where fewer than top_k can be chosen the
 * rest have index -1 and weight 0.
 *
 *   logits, type    tokens x experts, row pitch ldl, FP32 / BF16 / FP16
 *                   (gemm_out_t); computed in FP32
 *   bias            experts floats or NULL
 *   indices         tokens x top_k int32, dense
 *   weights         tokens x top_k float, dense
 *   offsets         experts + 1 int32: expert e has rows
 *                   [offsets[e], offsets[e + 1])
 *   order           tokens * top_k int32: row -> pair (token * top_k + choice),
 *                   pairs ascending within an expert; -1 past the last row
 *   slots           tokens x top_k int32: pair -> row, -1 without an expert
 * offsets, order and slots are all NULL (weights and indices only) or all
 * given.  experts <= 1024, tokens * top_k < 2^31.
 */
GEMM_API int gemm_route(int64_t tokens, int64_t experts, int type, const void *logits, int64_t ldl, const float *bias,
                        const gemm_route_t *how, int32_t *indices, float *weights, int32_t *offsets, int32_t *order,
                        int32_t *slots, struct CUstream_st *stream);

/* gemm_route_backward -- the logits' gradient (tokens x experts of `type`, row
 * pitch ldd) from the weights' gradient `grad` (tokens x top_k float, dense)
 * and the indices gemm_route returned.  The choice itself has no gradient. */
GEMM_API int gemm_route_backward(int64_t tokens, int64_t experts, int type, const void *logits, int64_t ldl,
                                 const gemm_route_t *how, const int32_t *indices, const float *grad, void *dlogits,
                                 int64_t ldd, struct CUstream_st *stream);

/*
 * gemm_combine -- out[t][:] = sum_j weights[t][j] * Y[slots[t][j]][:] in FP32,
 * in the order of j, rounded once to `type`.
 *   Y, ldy     rows x hidden of `type`; slots outside [0, rows) add nothing
 *   weights    tokens x top_k float, dense, or NULL for ones (the gradient of
 *              a scatter of each token to its rows)
 */
GEMM_API int gemm_combine(int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows, int type, const void *Y,
                          int64_t ldy, const int32_t *slots, const float *weights, void *out, int64_t ldo,
                          struct CUstream_st *stream);

/*
 * gemm_combine_backward -- from grad (tokens x hidden, the gradient of out):
 *   dY[slots[t][j]][:] = weights[t][j] * grad[t][:]
 *   dweights[t][j]     = <grad[t], Y[slots[t][j]]>  (0 where there is no row)
 *   order      gemm_route's row -> pair array of tokens * top_k (= rows)
 *              entries, or NULL: rows with -1 get a zero gradient; with NULL,
 *              rows no slot names keep what they hold
 */
GEMM_API int gemm_combine_backward(int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows, int type,
                                   const void *grad, int64_t ldg, const void *Y, int64_t ldy, const int32_t *slots,
                                   const float *weights, const int32_t *order, void *dY, int64_t ldd,
                                   float *dweights, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* TCGEMM_GEMM_OPS_H */

/*
 * gemm_project.h -- C ABI of the products around a language model's weights in
 * 16 bits (libtcgemm.so): the loss of the output projection over a vocabulary,
 * without keeping the logits, with its gradients; and low-rank adapters of many
 * requests beside a shared projection, with theirs.
 *
 * Conventions are gemm.h's and gemm_ops.h's: device pointers owned by the caller,
 * leading dimensions and strides in ELEMENTS, work enqueued on the caller's stream
 * without synchronising, a gemm_status_t returned, gemm_last_error() for the
 * message.  `dtype` is GEMM_BF16 or GEMM_FP16 and holds for every matrix of a call
 * that has no type of its own.  Sums are FP32.  A kernel wait that runs out is
 * reported by gemm_get_status().
 */
#ifndef TCGEMM_GEMM_PROJECT_H
#define TCGEMM_GEMM_PROJECT_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Variants of the loss; all 0: plain softmax cross entropy. */
typedef struct {
    float softcap;     /* c > 0: logits are c * tanh(z / c); 0: z itself       */
    float smoothing;   /* s in [0, 1): the target is 1 - s on the label plus
                          s / V everywhere                                     */
    float z_loss;      /* a >= 0: a * lse^2 is added                           */
} gemm_loss_t;

/*
 * gemm_project_loss -- for every token t of H (T x D) and the vocabulary's rows
 * W (V x D), with z[t][v] = <H[t], W[v]> (capped):
 *
 *     lse[t]  = log sum_v exp(z[t][v])
 *     loss[t] = lse[t] - (1 - s) z[t][label[t]] - s/V sum_v z[t][v] + a lse[t]^2
 *
 * The logits stay on the chip: each tile's maximum, sum of exponentials (FP32),
 * sum and label logit are all that leaves it.  A label outside [0, V) marks a token
 * that does not count: its loss is 0, whatever H[t] holds; lse[t] is that row's
 * all the same.
 *
 *   H            row pitch ldh >= D (T > 1)
 *   W            w_major 0: V rows of D values, pitch ldw >= D; 1: D rows of V
 *                values, pitch ldw >= V (the matrix a projection C = H.W takes)
 *   labels       T integers of label_bytes (4 or 8) each
 *   how          NULL or the variant
 *   loss, lse    T floats each (loss may be NULL)
 */
GEMM_API int gemm_project_loss(int64_t T, int64_t V, int64_t D, int dtype, const void *H, int64_t ldh, const void *W,
                               int64_t ldw, int w_major, const void *labels, int label_bytes, const gemm_loss_t *how,
                               float *loss, float *lse, struct CUstream_st *stream);

/*
 * gemm_project_loss_backward -- the gradients of H and W from grad[t], the
 * gradient of loss[t]:
 *
 *     d[t][v] = grad[t] ((1 + 2 a lse[t]) p[t][v] - (1 - s) [v = label] - s/V)
 *               * (1 - (z / c)^2 if capped),        p = exp(z - lse[t])
 *     dH = d . W,    dW = d^T . H
 *
 * The vocabulary is taken in pieces: a piece's logits are computed again, their
 * gradient d is rounded to `dtype` (with FP16 scaled by a power of two so that the
 * largest fits and the small ones keep their digits) and goes into both products;
 * dH is summed over the pieces in FP32.  What rounding takes from a row's largest
 * entry, the label's, is added back in FP32.  A token without a label adds nothing,
 * whatever H[t] and grad[t] hold, and gets a zero row in dH (W must be finite).
 *
 *   grad         T floats, grad_stride (0: one value for all, or 1) apart
 *   lse          as gemm_project_loss returned it for the same arguments
 *   dH           T x D, pitch lddh, or NULL
 *   dW           as W lies (w_major), pitch lddw, or NULL
 */
GEMM_API int gemm_project_loss_backward(int64_t T, int64_t V, int64_t D, int dtype, const float *grad,
                                        int64_t grad_stride, const void *H, int64_t ldh, const void *W, int64_t ldw,
                                        int w_major, const void *labels, int label_bytes, const gemm_loss_t *how,
                                        const float *lse, void *dH, int64_t lddh, void *dW, int64_t lddw,
                                        struct CUstream_st *stream);

/*
 * gemm_adapter_plan -- which tokens take which adapter, in the form the products
 * below read it.  ids: T int32, token t takes adapter ids[t]; values outside
 * [0, adapters) take none.  Tokens may come in any order; the products cost least
 * when neighbours share an adapter, for the tokens of a granule (16 to 256 neighbours)
 * take the products of all its adapters.  One plan serves every projection of a step.
 *
 *   plan         gemm_adapter_plan_words(T, adapters, backward) int32 words
 *   backward     1: with what gemm_adapters_backward needs besides
 *
 * T is at most 2^23 and adapters at most 4096 (gemm_adapter_plan_words: -1 beyond).
 */
GEMM_API int64_t gemm_adapter_plan_words(int64_t T, int64_t adapters, int backward);
GEMM_API int gemm_adapter_plan(int64_t T, int64_t adapters, const int32_t *ids, int backward, int32_t *plan,
                               struct CUstream_st *stream);

/* A stack of adapters: `count` pairs of rank x K (A) and rank x N (B) matrices, rows
 * of A and of B lda and ldb apart, matrices a_stride and b_stride.  Bases, pitches
 * and strides are multiples of 16 bytes (else GEMM_ERR_UNSUPPORTED), values finite:
 * the tokens of a tile share the products of its adapters, each taking its own, so
 * an infinity in one adapter would reach its neighbours' tokens.  rank is in
 * [1, 128].  scales: count floats on the device, or NULL (ones). */
typedef struct {
    int64_t count, rank;
    const void *A;
    int64_t lda, a_stride;
    const void *B;
    int64_t ldb, b_stride;
    const float *scales;
} gemm_adapters_t;

/*
 * gemm_adapters -- for every token t with adapter i:
 *
 *     C[t] = act(X[t] . W + scales[i] (X[t] . A_i^T) . B_i + bias)
 *
 * and without the middle term for a token that takes none.  The rank-wide
 * X[t] . A_i^T is scaled and rounded to `dtype` once (up to 32 tokens: to two numbers
 * of `dtype`, the second what the first left; in FP16 it has to stay below 65504);
 * everything else is FP32 up to the one
 * rounding of C.  The workspace is T x min(256, count) x the rank rounded up to 16,
 * 32, 64 or 128, in 16 bits (twice that up to 32 tokens, four times for the gradients).
 *
 *   X            T x K, pitch ldx >= K
 *   W            w_major 0: K rows of N values, pitch ldw >= N; 1: N rows of K,
 *                pitch ldw >= K.  Base and pitch multiples of 16 bytes.
 *   plan         gemm_adapter_plan's for T and count
 *   epi          NULL (C of `dtype`) or bias, act and C's type; alpha 1, beta 0.
 *                The activations keep a NaN.
 */
GEMM_API int gemm_adapters(int64_t T, int64_t N, int64_t K, int dtype, const void *X, int64_t ldx, const void *W,
                           int64_t ldw, int w_major, const gemm_adapters_t *adapters, const int32_t *plan, void *C,
                           int64_t ldc, const gemm_epilogue_t *epi, struct CUstream_st *stream);

/*
 * gemm_adapters_backward -- the gradients of X and of every adapter from dY, the
 * gradient of C without bias and activation (W is taken as frozen):
 *
 *     dX[t]  = dY[t] . W^T + scales[i] (dY[t] . B_i^T) . A_i
 *     dA_i   = sum_t (scales[i] dY[t] . B_i^T)^T X[t]      over the tokens of i
 *     dB_i   = sum_t (scales[i] X[t] . A_i^T)^T dY[t]
 *
 * In dA and dB the rank-wide factors are two numbers of `dtype` each, as above.
 *
 *   plan         made with backward = 1
 *   dX           T x K, pitch lddx, or NULL
 *   dA, dB       count x rank x K and count x rank x N without gaps, or NULL; zero
 *                for an adapter without tokens
 *
 * X's and dY's rows must be finite where any adapter is trained: a token adds a zero
 * multiple of its row to the adapters of its neighbours.
 */
GEMM_API int gemm_adapters_backward(int64_t T, int64_t N, int64_t K, int dtype, const void *dY, int64_t ldy,
                                    const void *X, int64_t ldx, const void *W, int64_t ldw, int w_major,
                                    const gemm_adapters_t *adapters, const int32_t *plan, void *dX, int64_t lddx,
                                    void *dA, void *dB, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif
#endif /* TCGEMM_GEMM_PROJECT_H */

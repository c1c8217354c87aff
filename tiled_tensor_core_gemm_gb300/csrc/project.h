// The 16-bit product kernel behind the output projection's loss and the low-rank
// adapters (project.cu), as their C entries (loss.cu, adapter.cu) call it.
#pragma once

#include "ops.h"

namespace tcgemm {

// One operand: `rows` (the extent along the result's lanes or columns) x k, in
// either major.  ld: elements between rows (K-major) or between values of k.
struct ProductOperand {
    const void *p = nullptr;
    int64_t rows = 0, ld = 0;
    int mn = 0;                // 1: `rows` is the contiguous dimension
};

// The adapters' stack of matrices, each rank x cols, and the plan that says which
// tokens take which.
struct ProductAdapters {
    const void *p = nullptr;
    int64_t rank = 0, cols = 0, ld = 0, stride = 0, count = 0;
    int pitch = 0;             // rows a slot takes: the rank rounded up to 16, 32, 64 or 128
    int granule = 0;           // tokens that share a list of slots
    int max_slots = 0;
    const int32_t *slots = nullptr;      // [granule][max_slots]: the adapters in it
    const int32_t *counts = nullptr;     // [granule]
    const int32_t *slot_of = nullptr;    // [token]: its slot, -1 without an adapter
    const int32_t *lists = nullptr;      // [adapter][granules]: granule * 256 + slot of those that have it
    const int32_t *list_counts = nullptr;
    int64_t granules = 0;
    const float *scales = nullptr;       // [adapter] or nullptr
    void *low = nullptr;                 // tokens x (max_slots * pitch): the rank-wide activations,
    int64_t ld_low = 0;                  // zero in the slots that are not a token's; and, with
    int64_t rest = 0;                    // `rest` != 0, that many elements on, what their rounding took
};

// What the loss epilogues take and give, per token (lane).
struct ProductLoss {
    const void *labels = nullptr;
    int label_bytes = 8;
    int64_t first = 0;         // this call's first column of the whole vocabulary
    float softcap = 0.f, eps_v = 0.f, one_eps = 1.f;   // smoothing / vocab, 1 - smoothing
    int want_sum = 0;          // label smoothing: the sum of the logits too
    float2 *parts = nullptr;   // [part][token]: maximum (in base 2) and sum of the exponentials
    float *sums = nullptr;     // [part][token]
    float *hits = nullptr;     // [token]: the label's logit
    const float4 *rows = nullptr;   // [token]: lse in base 2, two factors (loss.cu), and 0 for one that
                                    // does not count, else 1
    float *rests = nullptr;         // [token]: what rounding took from the label's gradient
};

// The label entries of d are by far its largest, so their rounding would be nearly all
// of the gradients' error.  What it took (`rests`) is added back in FP32 where the
// products that read d are written: to dH the token's rest times its label's row of W,
// to dW the sum over the tokens that have the label of their rests times their rows of
// H (loss.cu: loss_rests, loss_rests_join).
struct ProductRests {
    int kind = 0;                   // 1: lanes are tokens; 2: lanes, 3: columns are the vocabulary
    int64_t ld = 0;
    // kind 1: by token, and rows of W by label or by token (of the piece, `cols` entries)
    const float *rests = nullptr;
    const void *w = nullptr;
    int by_token = 0;
    int64_t cols = 0;
    // kinds 2, 3: the row of `sums` of each entry of the vocabulary, -1 without a token
    const int32_t *index = nullptr;
    const float *sums = nullptr;
};

enum ProductMode : int {
    kModePlain = 0,            // D = P Q^T
    kModeAdd = 1,              // the same plus low x adapters: further K-blocks
    kModeLow = 2,              // low = tokens x adapters^T, masked (swapped)
    kModeGradient = 3          // one product per adapter over the tokens that take it (swapped)
};
enum ProductEpilogue : int { kEpiSwapped = 0, kEpiRows = 1, kEpiStats = 2, kEpiDlogits = 3,
                            kEpiRests = 4 /* kEpiRows with ProductRests */,
                            kEpiGradient = 5 /* kEpiSwapped of kModeGradient */ };

// Columns of the tile, CTAs of it, its K ranges within a cluster (swapped) or through
// memory (row-wise).
struct ProductPlan {
    int bn = 0, cg = 1, splits = 1, parts = 1;
    int p_rows = 128;          // rows of P a CTA loads: 128, or (statistics of few tokens) 32
    int width = 0;             // statistics: columns a tile covers, up to bn (0: bn)
};

struct ProductCall {
    int mode = kModePlain, epilogue = kEpiRows;
    int type = GEMM_OUT_BF16;              // of the operands
    int64_t I = 0, J = 0, K = 0;           // lanes, columns, sum
    ProductOperand p, q;
    ProductPlan plan;
    ProductAdapters ad;
    ProductLoss loss;
    ProductRests rests;
    void *C = nullptr;                     // swapped: C's columns are the lanes
    int64_t ldc = 0;
    int64_t c_stride = 0;                  // kModeGradient: between adapters' results
    int64_t part_rows = 0;                 // plan.parts > 1: rows of C between the ranges' sums,
                                           // at least I rounded up to 256
    bool padded = false;                   // C's rows have room for 64 columns at a time
    EpiParams epi;
    const float *old = nullptr;            // FP32 sums to add (row-wise epilogue), pitch ld_old
    int64_t ld_old = 0;
    const float *alpha = nullptr;          // a factor on the device, on top of epi.alpha
    // kModeLow and kModeGradient: a second product of the same kind in the same launch (the
    // two sides of a backward pass): tokens' activations `second`, their width `second_k`;
    // low: the adapters' other stack, `ad2.p`; both: C2 and its pitches.
    bool two = false;
    ProductOperand second;
    int64_t second_k = 0;
    ProductAdapters ad2;
    void *C2 = nullptr;
    int64_t ldc2 = 0, c_stride2 = 0;
    bool early = false;                    // the launch before this one, on this stream and from
                                           // the same entry, only makes `low`
};

// Launches it.  Returns a gemm_status_t.
int product_launch(const ProductCall &call, int sms, cudaStream_t stream);

// Tiles and K ranges: see project.cu.
ProductPlan product_plan_rows(int64_t I, int64_t J, int64_t K, int sms, int most_parts = 1);
ProductPlan product_plan_tokens(int64_t tokens, int64_t cols, int64_t K, int sms);

ProductPlan product_plan_low(int64_t tokens, int64_t lanes, int64_t K, int sms);
ProductPlan product_plan_gradient(int64_t pitch, int64_t adapters, int64_t cols, int64_t tokens, int sms);

// The same for the loss statistics; `any`: tiles may be of any width (W K-major).
ProductPlan product_plan_stats(int64_t tokens, int64_t vocab, int64_t K, bool any, int sms);

// Parts of the loss statistics that `cols` columns give.
int64_t product_parts(const ProductPlan &plan, int64_t cols);

inline int64_t op_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t op_round_up(int64_t a, int64_t b) { return op_cdiv(a, b) * b; }

}  // namespace tcgemm

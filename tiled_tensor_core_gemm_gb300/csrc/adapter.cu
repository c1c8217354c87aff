// Low-rank adapters of many requests beside a shared projection: the plan of which
// tokens take which adapter, and the C entries that put the products of project.cu
// together.
//
// C = X W + s (X A_i^T) B_i takes two launches: `low`, the rank-wide activations of
// every token in the slot of its adapter (X once for every 128 lanes of slots x rank of a
// tile's tokens, the adapters in use once a tile), and the projection, whose K-blocks go
// on over the slots of the tile's granule.  The projection does not wait for `low` until
// its own K-blocks are in.  What bounds it: the weight stream for few tokens (W, and the
// adapters in use once each), the tensor cores for many, where the slots add
// (slots x rank) / K to the projection's flops and as many again to low's: 8192 tokens
// over 64 adapters of rank 64, 4096 x 4096, take 199 us in the adapters' order and 635 in
// a random one (62 slots a granule).
#include <algorithm>

#include "gemm_project.h"
#include "project.h"

namespace tcgemm {
namespace {

constexpr int64_t kMaxTokens = 1 << 23;
constexpr int kMaxAdapters = 4096;

// Tokens that share a list of slots: a tile's tokens are all of one granule, so it
// is the widest tile taken for that many tokens.
int granule_of(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : T <= 512 ? 128 : 256; }

// A plan's arrays, in int32 words from its start.
struct PlanLayout {
    int granule, max_slots;
    int64_t granules, counts, slots, slot_of, list_counts, lists, words;
};

PlanLayout layout_of(int64_t T, int64_t L, int backward) {
    PlanLayout p;
    p.granule = granule_of(T);
    p.max_slots = (int)std::min<int64_t>(p.granule, L);
    p.granules = op_cdiv(T, p.granule);
    p.counts = 0;
    p.slots = p.counts + p.granules;
    p.slot_of = p.slots + p.granules * p.max_slots;
    p.list_counts = p.slot_of + T;
    p.lists = p.list_counts + (backward ? L : 0);
    p.words = p.lists + (backward ? L * p.granules : 0);
    return p;
}

// One granule a block, one token a thread: the adapters that occur, ascending, are
// its slots.
__global__ void __launch_bounds__(256)
plan_slots(int T, int L, int granule, int max_slots, const int32_t *__restrict__ ids, int32_t *counts, int32_t *slots,
           int32_t *slot_of) {
    pdl_enter();
    __shared__ uint32_t bits[kMaxAdapters / 32];
    __shared__ int before[kMaxAdapters / 32];
    const int words = (L + 31) / 32, i = threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * granule + i;
    for (int w = i; w < words; w += blockDim.x) bits[w] = 0u;
    __syncthreads();
    const int id = i < granule && t < T ? __ldg(ids + t) : -1;
    const bool some = id >= 0 && id < L;
    if (some) atomicOr(&bits[id >> 5], 1u << (id & 31));
    __syncthreads();
    if (i < 32) {
        int sum = 0;
        for (int w0 = 0; w0 < words; w0 += 32) {
            const int w = w0 + i, n = w < words ? __popc(bits[w]) : 0;
            int up = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, up, d);
                if (i >= d) up += x;
            }
            if (w < words) before[w] = sum + up - n;
            sum += __shfl_sync(0xffffffffu, up, 31);
        }
        if (i == 0) counts[blockIdx.x] = sum;
    }
    __syncthreads();
    int slot = -1;
    if (some) {
        slot = before[id >> 5] + __popc(bits[id >> 5] & ((1u << (id & 31)) - 1u));
        slots[(int64_t)blockIdx.x * max_slots + slot] = id;       // (the same from all its tokens)
    }
    if (i < granule && t < T) slot_of[t] = slot;
}

// One adapter a warp: the granules that have it, ascending, and its slot there.
__global__ void __launch_bounds__(256)
plan_lists(int L, int granules, int max_slots, const int32_t *__restrict__ counts, const int32_t *__restrict__ slots,
           int32_t *list_counts, int32_t *lists) {
    pdl_enter();
    const int a = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (a >= L) return;
    int32_t *list = lists + (int64_t)a * granules;
    int n = 0;
    for (int g0 = 0; g0 < granules; g0 += 32) {
        const int g = g0 + lane;
        int at = -1;
        if (g < granules) {
            const int32_t *s = slots + (int64_t)g * max_slots;
            int lo = 0, hi = counts[g];           // the first slot not below a
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s[mid] < a) lo = mid + 1;
                else hi = mid;
            }
            if (lo < counts[g] && s[lo] == a) at = lo;
        }
        const uint32_t found = __ballot_sync(0xffffffffu, at >= 0);
        if (at >= 0) list[n + __popc(found & ((1u << lane) - 1u))] = g * 256 + at;
        n += __popc(found);
    }
    if (lane == 0) list_counts[a] = n;
}

struct Side {                  // activations, T x cols
    const char *name;
    const void *p;
    int64_t cols, ld;
    bool pack;
    uint64_t lo, hi, at;
};

struct Stack {                 // the adapters' A or B
    const char *name;
    const void *p;
    int64_t cols, ld, stride;
};

int invalid(const char *msg) { return api_error(GEMM_ERR_INVALID_ARG, msg); }

int check_sizes(int64_t T, int64_t N, int64_t K, int dtype, int64_t ldw, int w_major, const gemm_adapters_t *ad, int *type) {
    const int64_t kMax = 0x7fffffffLL - 512, kLdMax = 1LL << 36;
    if (dtype != GEMM_BF16 && dtype != GEMM_FP16) return invalid("dtype must be BF16 or FP16");
    *type = dtype == GEMM_BF16 ? GEMM_OUT_BF16 : GEMM_OUT_F16;
    if (T < 0 || N < 0 || K < 0 || N > kMax || K > kMax) return invalid("size negative or out of range");
    if (T > kMaxTokens) return invalid("at most 2^23 tokens");
    if (w_major != 0 && w_major != 1) return invalid("w_major is 0 or 1");
    if (ldw < std::max<int64_t>(w_major ? K : N, 1) || ldw > kLdMax) return invalid("leading dimension of W out of range");
    if (!ad) return invalid("adapters is NULL");
    if (ad->count < 1 || ad->count > kMaxAdapters) return invalid("adapters must be in [1, 4096]");
    if (ad->rank < 1 || ad->rank > 128) return invalid("rank must be in [1, 128]");
    if (ad->lda < std::max<int64_t>(K, 1) || ad->ldb < std::max<int64_t>(N, 1) || ad->lda > kLdMax || ad->ldb > kLdMax ||
        (ad->count > 1 && (ad->a_stride < std::max<int64_t>(K, 1) || ad->b_stride < std::max<int64_t>(N, 1))) || ad->a_stride < 0 ||
        ad->b_stride < 0 || ad->a_stride > (1LL << 38) || ad->b_stride > (1LL << 38))
        return invalid("leading dimension or stride of the adapters out of range");
    return GEMM_OK;
}

uint64_t stack_bytes(const gemm_adapters_t *ad, int64_t cols, int64_t ld, int64_t stride) {
    return op_bytes({{ad->count, stride}, {ad->rank, ld}, {cols, 1}}, 2);
}

// Weights are laid out once: what TMA cannot address is refused.
int check_weights(const gemm_adapters_t *ad, int64_t T, int64_t N, int64_t K, const void *W, int64_t ldw, int64_t w_rows) {
    auto ok = [](const void *p, int64_t rows, int64_t ld) { return (uintptr_t)p % 16 == 0 && (rows <= 1 || ld % 8 == 0); };
    if (K == 0 || N == 0 || T == 0) return GEMM_OK;
    if (!ok(W, w_rows, ldw)) return api_error(GEMM_ERR_UNSUPPORTED, "W's base and pitch must be multiples of 16 bytes");
    if (!ok(ad->A, ad->rank, ad->lda) || !ok(ad->B, ad->rank, ad->ldb) ||
        (ad->count > 1 && (ad->a_stride % 8 != 0 || ad->b_stride % 8 != 0)))
        return api_error(GEMM_ERR_UNSUPPORTED, "the adapters' bases, pitches and strides must be multiples of 16 bytes");
    return GEMM_OK;
}

ProductAdapters adapters_of(const gemm_adapters_t *ad, const int32_t *plan, const PlanLayout &l) {
    ProductAdapters a;
    a.rank = ad->rank;
    a.count = ad->count;
    a.pitch = ad->rank <= 16 ? 16 : ad->rank <= 32 ? 32 : ad->rank <= 64 ? 64 : 128;
    a.granule = l.granule;
    a.max_slots = l.max_slots;
    a.granules = l.granules;
    a.counts = plan + l.counts;
    a.slots = plan + l.slots;
    a.slot_of = plan + l.slot_of;
    a.list_counts = plan + l.list_counts;
    a.lists = plan + l.lists;
    a.scales = ad->scales;
    a.ld_low = (int64_t)a.max_slots * a.pitch;
    return a;
}

// low = scale * x . stack_i^T, in the slot of each token's adapter; with x2 the same of
// it and stack2 to low2, in the same launch.
int run_low(int64_t T, int type, const Side &x, const Stack &stack, ProductAdapters ad, void *low, const Side *x2, const Stack *stack2,
            void *low2, int sms, cudaStream_t stream) {
    auto with = [](ProductAdapters a, const Stack &s) {
        a.p = s.p;
        a.cols = s.cols;
        a.ld = s.ld;
        a.stride = s.stride;
        return a;
    };
    ProductCall c;
    c.mode = kModeLow;
    c.epilogue = kEpiSwapped;
    c.type = type;
    c.I = ad.ld_low;
    c.J = T;
    c.K = x.cols;
    c.plan = product_plan_low(T, x2 ? 2 * op_round_up(ad.ld_low, 128) : ad.ld_low, x2 ? std::min(x.cols, x2->cols) : x.cols, sms);
    c.q = {x.p, T, x.ld, 0};
    c.ad = with(ad, stack);
    c.C = low;
    c.ldc = ad.ld_low;
    if (x2) {
        c.two = true;
        c.second = {x2->p, T, x2->ld, 0};
        c.second_k = x2->cols;
        c.ad2 = with(ad, *stack2);
        c.C2 = low2;
        c.ldc2 = ad.ld_low;
    }
    c.epi.active = 1;
    c.epi.out = type;
    return product_launch(c, sms, stream);
}

// C = act(x . W + low x stack + bias).  w_k_major: W's rows are the columns of C.  low_k: what
// the launch that makes low sums over, its two products' lengths together.
int run_add(int64_t T, int64_t cols, int type, const Side &x, const void *W, int64_t ldw, bool w_k_major, const Stack &stack,
            ProductAdapters ad, void *low, int64_t low_k, void *C, int64_t ldc, const EpiParams &epi, int sms, cudaStream_t stream) {
    ProductCall c;
    c.mode = kModeAdd;
    c.type = type;
    c.K = x.cols;
    const ProductPlan rows = product_plan_rows(T, cols, x.cols, sms), few = product_plan_tokens(T, cols, x.cols, sms);
    // Tokens on the columns while there are at most 128 of them, or while tiles of
    // 128 tokens with K ranges still fill the SMs in one round.
    const bool swap = T <= 128 || (T <= 512 && op_cdiv(cols, 128) * op_cdiv(T, 128) <= sms);
    c.epilogue = swap ? kEpiSwapped : kEpiRows;
    const ProductOperand w = {W, cols, ldw, w_k_major ? 0 : 1}, t = {x.p, T, x.ld, 0};
    c.plan = swap ? few : rows;
    if (!swap && ad.granule < 128 * c.plan.cg) c.plan.bn = 128, c.plan.cg = 1;
    c.I = swap ? cols : T;
    c.J = swap ? T : cols;
    c.p = swap ? w : t;
    c.q = swap ? t : w;
    ad.p = stack.p;
    ad.cols = stack.cols;
    ad.ld = stack.ld;
    ad.stride = stack.stride;
    ad.low = low;
    c.ad = ad;
    c.C = C;
    c.ldc = ldc;
    c.epi = epi;
    // Where low may take long its end is waited for first: the MMAs' wait for a slot of it is
    // bounded by the option.  At 64 x 128 x 64 multiply-adds in 0.18 us an SM (project.cu) the
    // rule gives low's launch a seventeenth of the limit.
    c.early = (double)T * (double)ad.ld_low * (double)low_k < 2.5e10 * options_snapshot().wait_timeout_ms;
    return product_launch(c, sms, stream);
}

// For each adapter low^T . x over its tokens, rank x cols: dA from up and X, dB from low
// and dY, in one launch where both are wanted.
int run_gradients(int64_t T, int type, ProductAdapters ad, const Side &x, void *up, void *dA, const Side &g, void *low, void *dB,
                  int sms, cudaStream_t stream) {
    const Side &one = dA ? x : g;
    ProductCall c;
    c.mode = kModeGradient;
    c.epilogue = kEpiGradient;
    c.type = type;
    c.I = one.cols;
    c.J = ad.rank;
    c.K = T;
    c.plan = product_plan_gradient(ad.pitch, ad.count, one.cols + (dA && dB ? op_round_up(g.cols, 128) : 0), T, sms);
    c.p = {one.p, one.cols, one.ld, 1};
    c.q.mn = 1;                                   // (low, from its own map)
    c.ad = ad;
    c.ad.low = dA ? up : low;
    c.C = dA ? dA : dB;
    c.ldc = one.cols;
    c.c_stride = ad.rank * one.cols;
    if (dA && dB) {
        c.two = true;
        c.second = {g.p, g.cols, g.ld, 1};
        c.second_k = g.cols;
        c.ad2 = ad;
        c.ad2.low = low;
        c.C2 = dB;
        c.ldc2 = g.cols;
        c.c_stride2 = ad.rank * g.cols;
    }
    c.epi.active = 1;
    c.epi.out = type;
    return product_launch(c, sms, stream);
}

// Whether the activations have to be copied, and where to.
int plan_side(Side *s, int64_t T, int dev, uint64_t *bytes) {
    if (T <= 1) s->ld = op_round_up(std::max<int64_t>(s->cols, 1), 8);
    s->pack = s->cols > 0 && !op_wide(s->p, s->ld, 2);
    s->at = *bytes;
    if (!s->pack) return GEMM_OK;
    *bytes += ((uint64_t)T * op_round_up(s->cols, 8) * 2 + 255) / 256 * 256;
    return api_check_device_span_range(s->name, s->p, op_extent(T, s->cols, s->ld, 2), dev, &s->lo, &s->hi);
}

int pack_side(Side *s, int64_t T, uint8_t *base, cudaStream_t stream) {
    if (!s->pack) return GEMM_OK;
    const int64_t ld = op_round_up(s->cols, 8);
    const int rc = op_launched("operand pack", pack_rows_launch(s->p, s->ld, base + s->at, ld, T, s->cols, 2, s->lo, s->hi, stream));
    s->p = base + s->at;
    s->ld = ld;
    return rc;
}

int workspace(void **ws, uint64_t bytes, int dev, cudaStream_t stream) {
    const cudaError_t e = op_malloc(ws, bytes, dev, stream);
    if (e == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    char msg[128];
    std::snprintf(msg, sizeof msg, "workspace of %llu bytes: %s", (unsigned long long)bytes, cudaGetErrorString(e));
    return api_error(GEMM_ERR_NO_MEMORY, msg);
}

}  // namespace
}  // namespace tcgemm

using namespace tcgemm;

extern "C" {

int64_t gemm_adapter_plan_words(int64_t T, int64_t adapters, int backward) {
    if (T < 0 || T > kMaxTokens || adapters < 1 || adapters > kMaxAdapters) return -1;
    return layout_of(T, adapters, backward).words;
}

int gemm_adapter_plan(int64_t T, int64_t adapters, const int32_t *ids, int backward, int32_t *plan, struct CUstream_st *stream_) {
    api_clear_error();
    if (gemm_adapter_plan_words(T, adapters, backward) < 0) return invalid("tokens must be in [0, 2^23], adapters in [1, 4096]");
    const PlanLayout l = layout_of(T, adapters, backward);
    OpSpan spans[2] = {{"ids", ids, (uint64_t)T * 4, 4, false}, {"plan", plan, (uint64_t)l.words * 4, 4, true}};
    if (l.words == 0) return GEMM_OK;
    int rc = op_check(spans, 2, nullptr);
    if (rc) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T > 0)
        rc = op_launched("adapter plan", launch_pdl(plan_slots, dim3((unsigned)l.granules), dim3(l.granule < 32 ? 32 : l.granule), 0,
                                                    stream, (int)T, (int)adapters, l.granule, l.max_slots, ids, plan + l.counts,
                                                    plan + l.slots, plan + l.slot_of));
    if (rc == GEMM_OK && backward)
        rc = op_launched("adapter lists",
                         launch_pdl(plan_lists, dim3((unsigned)op_cdiv(adapters, 8)), dim3(256), 0, stream, (int)adapters,
                                    (int)l.granules, l.max_slots, (const int32_t *)(plan + l.counts),
                                    (const int32_t *)(plan + l.slots), plan + l.list_counts, plan + l.lists));
    return rc;
}

int gemm_adapters(int64_t T, int64_t N, int64_t K, int dtype, const void *X, int64_t ldx, const void *W, int64_t ldw, int w_major,
                  const gemm_adapters_t *ad, const int32_t *plan, void *C, int64_t ldc, const gemm_epilogue_t *epi_in,
                  struct CUstream_st *stream_) {
    api_clear_error();
    int type = 0, rc = check_sizes(T, N, K, dtype, ldw, w_major, ad, &type);
    if (rc) return rc;
    EpiParams epi;
    if ((rc = api_epilogue(epi_in, &epi))) return rc;
    if (!epi_in) epi.out = type;
    if (epi.alpha != 1.f || epi.beta != 0.f) return invalid("gemm_adapters takes alpha = 1 and beta = 0");
    if (!epi.active) epi.act = GEMM_ACT_NONE, epi.bias = nullptr;
    epi.active = 1;
    const int64_t kLdMax = 1LL << 36;
    if (ldx < std::max<int64_t>(K, 1) || ldc < std::max<int64_t>(N, 1) || ldx > kLdMax || ldc > kLdMax)
        return invalid("leading dimension out of range");
    const int ob = op_type_bytes(epi.out);
    const PlanLayout l = layout_of(T, ad->count, 0);
    OpSpan spans[8] = {{"X", X, op_extent(T, K, ldx, 2), 2, false},
                       {"W", W, w_major ? op_extent(N, K, ldw, 2) : op_extent(K, N, ldw, 2), 2, false},
                       {"A", ad->A, stack_bytes(ad, K, ad->lda, ad->a_stride), 2, false},
                       {"B", ad->B, stack_bytes(ad, N, ad->ldb, ad->b_stride), 2, false},
                       {"scales", ad->scales, ad->scales ? (uint64_t)ad->count * 4 : 0, 4, false},
                       {"plan", plan, (uint64_t)l.words * 4, 4, false},
                       {"bias", epi.bias, epi.bias ? (uint64_t)N * 4 : 0, 4, false},
                       {"C", C, op_extent(T, N, ldc, ob), ob, true}};
    if (T == 0 || N == 0) return GEMM_OK;
    if ((rc = check_weights(ad, T, N, K, W, ldw, w_major ? N : K))) return rc;
    int sms = 0;
    if ((rc = op_check(spans, 8, &sms))) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    cudaGetDevice(&dev);
    ProductAdapters pa = adapters_of(ad, plan, l);
    Side x = {"X", X, K, ldx, false, 0, 0, 0};
    // Few tokens do not average low's rounding out, and their tiles have room for the rests.
    if (T <= 32) pa.rest = T * pa.ld_low;
    uint64_t bytes = ((uint64_t)T * pa.ld_low * (pa.rest ? 4 : 2) + 255) / 256 * 256;
    if ((rc = plan_side(&x, T, dev, &bytes))) return rc;
    void *ws = nullptr;
    if ((rc = workspace(&ws, bytes, dev, stream))) return rc;
    rc = pack_side(&x, T, static_cast<uint8_t *>(ws), stream);
    const Stack a = {"A", ad->A, K, ad->lda, ad->a_stride}, b = {"B", ad->B, N, ad->ldb, ad->b_stride};
    if (rc == GEMM_OK) rc = run_low(T, type, x, a, pa, ws, nullptr, nullptr, nullptr, sms, stream);
    if (rc == GEMM_OK) rc = run_add(T, N, type, x, W, ldw, w_major != 0, b, pa, ws, K, C, ldc, epi, sms, stream);
    const cudaError_t e = cudaFreeAsync(ws, stream);
    return rc ? rc : op_launched("cudaFreeAsync", e);
}

int gemm_adapters_backward(int64_t T, int64_t N, int64_t K, int dtype, const void *dY, int64_t ldy, const void *X, int64_t ldx,
                           const void *W, int64_t ldw, int w_major, const gemm_adapters_t *ad, const int32_t *plan, void *dX,
                           int64_t lddx, void *dA, void *dB, struct CUstream_st *stream_) {
    api_clear_error();
    int type = 0, rc = check_sizes(T, N, K, dtype, ldw, w_major, ad, &type);
    if (rc) return rc;
    const int64_t kLdMax = 1LL << 36;
    if (ldx < std::max<int64_t>(K, 1) || ldy < std::max<int64_t>(N, 1) || ldx > kLdMax || ldy > kLdMax ||
        (dX && (lddx < std::max<int64_t>(K, 1) || lddx > kLdMax)))
        return invalid("leading dimension out of range");
    const PlanLayout l = layout_of(T, ad->count, 1);
    const uint64_t da = dA ? op_bytes({{ad->count * ad->rank, K}, {K, 1}}, 2) : 0, db = dB ? op_bytes({{ad->count * ad->rank, N}, {N, 1}}, 2) : 0;
    OpSpan spans[10] = {{"dY", dY, op_extent(T, N, ldy, 2), 2, false},
                        {"X", X, dA || dB ? op_extent(T, K, ldx, 2) : 0, 2, false},
                        {"W", W, !dX ? 0 : w_major ? op_extent(N, K, ldw, 2) : op_extent(K, N, ldw, 2), 2, false},
                        {"A", ad->A, stack_bytes(ad, K, ad->lda, ad->a_stride), 2, false},
                        {"B", ad->B, stack_bytes(ad, N, ad->ldb, ad->b_stride), 2, false},
                        {"scales", ad->scales, ad->scales ? (uint64_t)ad->count * 4 : 0, 4, false},
                        {"plan", plan, (uint64_t)l.words * 4, 4, false},
                        {"dX", dX, dX ? op_extent(T, K, lddx, 2) : 0, 2, true},
                        {"dA", dA, da, 2, true},
                        {"dB", dB, db, 2, true}};
    if (!dX && !dA && !dB) return GEMM_OK;
    if ((rc = check_weights(ad, T, N, K, dX ? W : nullptr, dX ? ldw : 8, w_major ? N : K))) return rc;
    int sms = 0;
    if ((rc = op_check(spans, 10, &sms))) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T == 0) {
        if (da) rc = op_launched("cudaMemsetAsync", cudaMemsetAsync(dA, 0, da, stream));
        if (rc == GEMM_OK && db) rc = op_launched("cudaMemsetAsync", cudaMemsetAsync(dB, 0, db, stream));
        return rc;
    }
    int dev = 0;
    cudaGetDevice(&dev);
    ProductAdapters pa = adapters_of(ad, plan, l);
    Side x = {"X", X, K, ldx, false, 0, 0, 0}, g = {"dY", dY, N, ldy, false, 0, 0, 0};
    const bool want_up = (dX && K > 0) || da, want_low = db != 0;
    pa.rest = T * pa.ld_low;
    const uint64_t low_bytes = ((uint64_t)T * pa.ld_low * 4 + 255) / 256 * 256;
    uint64_t bytes = low_bytes * ((want_up ? 1 : 0) + (want_low ? 1 : 0));
    if (bytes == 0) return GEMM_OK;
    if ((rc = plan_side(&g, T, dev, &bytes))) return rc;
    if ((da || db) && (rc = plan_side(&x, T, dev, &bytes))) return rc;
    void *ws = nullptr;
    if ((rc = workspace(&ws, bytes, dev, stream))) return rc;
    uint8_t *base = static_cast<uint8_t *>(ws), *up = base, *low = base + (want_up ? low_bytes : 0);
    const Stack a = {"A", ad->A, K, ad->lda, ad->a_stride}, b = {"B", ad->B, N, ad->ldb, ad->b_stride};
    rc = pack_side(&g, T, base, stream);
    if (rc == GEMM_OK) rc = pack_side(&x, T, base, stream);
    if (rc == GEMM_OK) {
        if (want_up && want_low) rc = run_low(T, type, g, b, pa, up, &x, &a, low, sms, stream);
        else rc = want_up ? run_low(T, type, g, b, pa, up, nullptr, nullptr, nullptr, sms, stream)
                          : run_low(T, type, x, a, pa, low, nullptr, nullptr, nullptr, sms, stream);
    }
    if (rc == GEMM_OK && dX && K > 0) {
        EpiParams epi;
        epi.active = 1;
        epi.out = type;
        rc = run_add(T, K, type, g, W, ldw, w_major == 0, a, pa, up, N + (want_low ? K : 0), dX, lddx, epi, sms, stream);
    }
    if (rc == GEMM_OK && (da || want_low))
        rc = run_gradients(T, type, pa, x, up, da ? dA : nullptr, g, low, want_low ? dB : nullptr, sms, stream);
    const cudaError_t e = cudaFreeAsync(ws, stream);
    return rc ? rc : op_launched("cudaFreeAsync", e);
}

}  // extern "C"

// Routing of tokens to experts: scores, groups, the top_k largest, weights, and
// the (token, choice) pairs in expert order; and the logits' gradient.
//
//   s = softmax(x) or 1 / (1 + exp(-x)),  key = s + b (x itself without b),
//   w_j = scale * s_j / sum_i s_i  over the chosen experts (or scale * s_j).
//   ds_j = scale * (g_j - sum_i g_i s_i / Z) / Z, Z = sum_i s_i (or scale * g_j),
//   dx = s * (ds - sum ds * s)  (softmax)  or  ds * s(x) * s(-x)  (sigmoid).
//
// One warp takes a token and holds its row in registers, four neighbouring
// experts a lane and step.  Keys are compared as unsigned integers in the order
// of the floats, so a warp's largest is one redux and its lowest index another;
// 0 is kept for "cannot be chosen".  Scores are computed with the full-range
// expf and IEEE divisions: the choice hangs on their last bits, so approximate
// ones would choose differently from the formulas more often.
//
// The order by expert is a counting sort without atomics on global memory, so
// it does not depend on timing: a block takes 32 neighbouring tokens and keeps
// one word an expert in shared memory, bit t set when token t chose it; a pair's
// rank in the block is a population count, the block's counts go to a table,
// a second kernel scans the table's rows (one per expert, over the blocks) and
// a third adds the experts' offsets.  Up to kClusterTokens tokens the blocks of
// one cluster, 16 tokens each, read one another's counts in shared memory and
// do all of it in one launch.
//
// Bound by latency and issue, not by memory.  Measured on GB300: 48 x 256 with
// groups 11.5 us, one launch; 16384 x 128 16 us for the choice (4.2 MB of logits),
// 3.6 for the scan and 5 for the placing, 9.5 for the gradient.
#include <type_traits>

#include "ops.h"
#include "ptx_ops.cuh"

namespace tcgemm {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxGroups = 32;
constexpr int kMaxTopK = 32;
constexpr int kChunkTokens = 32;       // tokens of a block: bits of a word
constexpr int kWarps = 16;             // of a routing block
constexpr int kClusterTokens = 128;    // tokens one cluster routes and orders in one launch

struct RouteParams {
    const void *logits;
    int64_t ldl;
    const float *bias;
    int32_t *indices;
    float *weights;
    int32_t *offsets, *order, *slots;   // all or none
    int32_t *table;                     // [experts][blocks] counts, then first ranks; then [experts] totals
    int tokens, experts, blocks;
    int top_k, score, groups, per, top_groups, top2, renormalize;
    float scale;
    int wide;                           // rows are whole 4-element vectors
    // backward
    const float *grad;
    void *dlogits;
    int64_t ldd;
    int d_wide;
};

// Floats as unsigned integers in the same order (-0 as +0); NaN and -inf, which
// cannot be chosen, as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if (!(x > -INFINITY)) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Expert of a lane's i-th value.
__device__ __forceinline__ int expert_of(int i, int lane) { return (i >> 2) * 128 + lane * 4 + (i & 3); }

// A token's logits in FP32; -inf past the last expert and where the logit is NaN.
template <typename T, int EPL>
__device__ __forceinline__ void load_row(const T *row, int experts, int lane, bool wide, float (&x)[EPL]) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const int e = expert_of(i, lane);
        if (wide && e < experts) {
            struct alignas(4 * sizeof(T)) V4 { T v[4]; };
            const V4 v = *reinterpret_cast<const V4 *>(row + e);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] = OpType<T>::up(v.v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] = e + k < experts ? OpType<T>::up(row[e + k]) : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (!(x[i + k] > -INFINITY)) x[i + k] = -INFINITY;
    }
}

// From the shared memory of a block of the cluster (a shared::cluster address).
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// exp(x - m), m the row's largest; masked experts (-inf) have 0.  An infinite
// logit takes its limit: the softmax is shared by the infinite ones.
__device__ __forceinline__ float softmax_term(float x, float m) {
    if (!(x > -INFINITY)) return 0.f;
    return m == INFINITY ? (x == INFINITY ? 1.f : 0.f) : expf(x - m);
}

// An expert's score; z: the sum of the row's terms (softmax).
__device__ __forceinline__ float score_of(int score, float x, float m, float z) {
    if (!(x > -INFINITY)) return 0.f;
    return score == GEMM_SCORE_SIGMOID ? 1.f / (1.f + expf(-x)) : softmax_term(x, m) / z;
}

// Clears the keys of the experts whose group does not take part.  `v`: what the groups are
// judged by (keys, or scores where there is no bias), masked experts -inf; it
// goes through the warp's `buf` (padded one word in 32).  lanes: 32 over the
// power of two at or above the number of groups; `lanes` neighbouring lanes scan one group.
template <int EPL>
__device__ __forceinline__ void keep_groups(const RouteParams &p, const float (&v)[EPL], uint32_t (&key)[EPL], float *buf,
                                            int lane) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = expert_of(i, lane);
        if (e < p.experts) buf[e + (e >> 5)] = v[i];
    }
    __syncwarp();
    int pow2 = 1;
    while (pow2 < p.groups) pow2 <<= 1;
    const int lanes = 32 / pow2, g = lane / lanes, sub = lane & (lanes - 1);
    float a = -INFINITY, b = -INFINITY;      // the two largest
    if (g < p.groups)
        for (int i = sub; i < p.per; i += lanes) {
            const int e = g * p.per + i;
            const float y = buf[e + (e >> 5)];
            b = fmaxf(b, fminf(a, y));
            a = fmaxf(a, y);
        }
    __syncwarp();
    for (int o = 1; o < lanes; o <<= 1) {
        const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmaxf(fmaxf(b, b2), fminf(a, a2));
        a = fmaxf(a, a2);
    }
    if (p.top2 && b > -INFINITY) a = a + b;
    const uint32_t mine = g < p.groups ? key_of(a) : 0u;
    int ahead = 0;
    for (int o = 0; o < p.groups; ++o) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, o * lanes);
        ahead += other > mine || (other == mine && o < g);
    }
    const uint32_t keep = __ballot_sync(0xffffffffu, sub == 0 && mine != 0u && ahead < p.top_groups);
    uint32_t bits = 0;
    for (int o = 0; o < p.groups; ++o) bits |= ((keep >> (o * lanes)) & 1u) << o;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = expert_of(i, lane);
        if (e < p.experts && !((bits >> (e / p.per)) & 1u)) key[i] = 0u;
    }
}

// The largest of a lane's keys and its place (the first of equals).
template <int EPL>
__device__ __forceinline__ void lane_best(const uint32_t (&key)[EPL], uint32_t &best, int &at) {
    best = key[0];
    at = 0;
#pragma unroll
    for (int i = 1; i < EPL; ++i)
        if (key[i] > best) {
            best = key[i];
            at = i;
        }
}

// Routes token t by one warp; lane j < top_k returns the j-th choice (or -1)
// and writes it with its weight.
template <typename T, int EPL>
__device__ __forceinline__ int route_token(const RouteParams &p, int t, float *buf, int lane) {
    float x[EPL];
    const T *logits = static_cast<const T *>(p.logits) + (int64_t)t * p.ldl;
    load_row<T, EPL>(logits, p.experts, lane, p.wide, x);
    const bool grouped = p.groups > 1 && p.top_groups < p.groups;
    const bool by_score = p.bias || (grouped && p.top2);      // the choice needs every expert's score
    uint32_t key[EPL];
    float m = 0.f, z = 1.f;                                   // of the softmax: largest logit, sum
    if (p.score == GEMM_SCORE_SOFTMAX) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) m = fmaxf(m, x[i]);
        m = warp_max(m);
        // (renormalised weights divide by the chosen scores' sum: the whole sum cancels)
        if (by_score || !p.renormalize) {
            z = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) z += softmax_term(x[i], m);
            z = warp_sum(z);
        }
    }
    if (by_score) {
        float v[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = expert_of(i, lane);
            const float s = score_of(p.score, x[i], m, z);
            v[i] = p.bias && x[i] > -INFINITY ? s + __ldg(p.bias + e) : x[i];
            key[i] = key_of(v[i]);
            if (!p.bias) v[i] = s;
            if (!key[i]) v[i] = -INFINITY;
        }
        if (grouped) keep_groups<EPL>(p, v, key, buf, lane);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = key_of(x[i]);
        if (grouped) keep_groups<EPL>(p, x, key, buf, lane);
    }
    // The largest key of all lanes' largest, top_k times.  A lane with few keys
    // has them sorted (stably: equal keys in the order of their experts) and drops
    // its first when it wins; one with many looks for its next.
    int mine = -1;
    uint32_t best;
    int at;
    uint32_t places = 0;                     // of the sorted keys, four bits each
    if constexpr (EPL <= 8) {
        int place[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) place[i] = i;
#pragma unroll
        for (int n = 0; n < EPL; ++n)
#pragma unroll
            for (int i = n & 1; i + 1 < EPL; i += 2) {
                const bool swap = key[i] < key[i + 1];
                const uint32_t hi = max(key[i], key[i + 1]), lo = min(key[i], key[i + 1]);
                const int first = swap ? place[i + 1] : place[i], second = swap ? place[i] : place[i + 1];
                key[i] = hi;
                key[i + 1] = lo;
                place[i] = first;
                place[i + 1] = second;
            }
#pragma unroll
        for (int i = 0; i < EPL; ++i) places |= (uint32_t)place[i] << (4 * i);
        best = key[0];
        at = place[0];
    } else {
        lane_best<EPL>(key, best, at);
    }
    for (int j = 0; j < p.top_k; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0u) break;
        const uint32_t have = __ballot_sync(0xffffffffu, best == top);
        const int e = expert_of(at, lane);
        int winner = __ffs(have) - 1;
        if (have & (have - 1)) {             // equal keys: the lowest expert's
            const int low = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)e : 0xffffffffu);
            winner = (low >> 2) & 31;
        }
        const int chosen = __shfl_sync(0xffffffffu, e, winner);
        if (lane == j) mine = chosen;
        if constexpr (EPL <= 8) {
            const bool won = lane == winner;
#pragma unroll
            for (int i = 0; i + 1 < EPL; ++i) key[i] = won ? key[i + 1] : key[i];
            key[EPL - 1] = won ? 0u : key[EPL - 1];
            places = won ? places >> 4 : places;
            best = key[0];
            at = (int)(places & 15u);
        } else if (lane == winner) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == at) key[i] = 0u;
            lane_best<EPL>(key, best, at);
        }
    }
    float w = 0.f;
    if (mine >= 0) w = score_of(p.score, OpType<T>::up(logits[mine]), m, z);
    if (p.renormalize) {
        const float sum = warp_sum(w);
        if (sum > 0.f) w = w / sum;
    }
    if (lane < p.top_k) {
        p.indices[(int64_t)t * p.top_k + lane] = mine;
        p.weights[(int64_t)t * p.top_k + lane] = w * p.scale;
    }
    return mine;
}

// Exclusive sum of v[0 .. n) in shared memory, in place, by a block of THREADS;
// v[n] gets the total.  n <= kMaxExperts.
template <int THREADS>
__device__ __forceinline__ void block_scan(int32_t *v, int n) {
    constexpr int PER = kMaxExperts / THREADS;
    __shared__ int32_t s_warp[THREADS / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t c[PER], sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = (int)threadIdx.x * PER + k;
        c[k] = i < n ? v[i] : 0;
        sum += c[k];
    }
    int32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int32_t at = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const int32_t y = s_warp[w];
        if (w < warp) at += y;
        total += y;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = (int)threadIdx.x * PER + k;
        if (i < n) v[i] = at;
        at += c[k];
    }
    if (threadIdx.x == 0) v[n] = total;
    __syncthreads();
}

// Few tokens: the blocks of one cluster, kWarps neighbouring tokens each, route
// them, read one another's counts and place the pairs.
template <typename T, int EPL>
__global__ void __launch_bounds__(kWarps * 32) route_cluster_kernel(const RouteParams p) {
    __shared__ uint32_t s_chose[EPL * 32];          // bit w: the block's w-th token chose the expert
    __shared__ int32_t s_first[EPL * 32 + 1];       // the experts' first rows
    __shared__ int32_t s_before[EPL * 32];          // pairs of the expert in the blocks before this one
    extern __shared__ float s_buf[];                // the warps' group buffers
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    for (int i = threadIdx.x; i < EPL * 32; i += blockDim.x) s_chose[i] = 0u;
    pdl_enter();
    __syncthreads();
    const int t = (int)rank * kWarps + warp;
    int mine = -1;
    if (t < p.tokens) {
        mine = route_token<T, EPL>(p, t, s_buf + warp * (EPL * 33), lane);
        if (mine >= 0) atomicOr(&s_chose[mine], 1u << warp);      // (bits: the order of arrival is nothing)
    }
    __syncwarp();
    ptx::cluster_sync();
    const uint32_t chose = ptx::smem_addr(s_chose);
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) {
        int before = 0, all = 0;
        for (uint32_t r = 0; r < gridDim.x; ++r) {
            const int c = __popc(ld_cluster_u32(ptx::mapa_shared(chose + 4u * (uint32_t)e, r)));
            if (r < rank) before += c;
            all += c;
        }
        s_before[e] = before;
        s_first[e] = all;
    }
    __syncthreads();
    block_scan<kWarps * 32>(s_first, p.experts);
    if (rank == 0)
        for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) p.offsets[e] = s_first[e];
    const int pairs = p.tokens * p.top_k;
    for (int r = s_first[p.experts] + (int)(rank * blockDim.x + threadIdx.x); r < pairs; r += (int)(gridDim.x * blockDim.x))
        p.order[r] = -1;
    if (t < p.tokens && lane < p.top_k) {
        int slot = -1;
        if (mine >= 0) {
            slot = s_first[mine] + s_before[mine] + __popc(s_chose[mine] & ((1u << warp) - 1u));
            p.order[slot] = t * p.top_k + lane;
        }
        p.slots[t * p.top_k + lane] = slot;
    }
    __syncwarp();
    ptx::cluster_sync();          // (no block leaves while another may read its shared memory)
}

// Routes a block's 32 tokens; leaves each pair's rank among the block's pairs of
// its expert in slots, and the block's counts in the table.
template <typename T, int EPL>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p) {
    __shared__ uint32_t s_chose[EPL * 32];
    extern __shared__ float s_buf[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < EPL * 32; i += blockDim.x) s_chose[i] = 0u;
    pdl_enter();
    __syncthreads();
    int mine[kChunkTokens / kWarps];
#pragma unroll
    for (int n = 0; n < kChunkTokens / kWarps; ++n) {
        const int t = blockIdx.x * kChunkTokens + n * kWarps + warp;
        mine[n] = -1;
        if (t < p.tokens) {
            mine[n] = route_token<T, EPL>(p, t, s_buf + warp * (EPL * 33), lane);
            if (mine[n] >= 0) atomicOr(&s_chose[mine[n]], 1u << (n * kWarps + warp));
        }
    }
    if (!p.offsets) return;
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
        p.table[(int64_t)e * p.blocks + blockIdx.x] = __popc(s_chose[e]);
#pragma unroll
    for (int n = 0; n < kChunkTokens / kWarps; ++n) {
        const int b = n * kWarps + warp, t = blockIdx.x * kChunkTokens + b;
        if (t < p.tokens && lane < p.top_k)
            p.slots[(int64_t)t * p.top_k + lane] = mine[n] >= 0 ? __popc(s_chose[mine[n]] & ((1u << b) - 1u)) : -1;
    }
}

// One warp per expert: its counts over the blocks become first ranks; its total
// goes past the table.
__global__ void __launch_bounds__(128) route_scan_kernel(const RouteParams p) {
    pdl_enter();
    const int e = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= p.experts) return;
    int32_t *row = p.table + (int64_t)e * p.blocks;
    int32_t carry = 0;
    for (int i0 = 0; i0 < p.blocks; i0 += 128) {
        int32_t c[4], sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + lane * 4 + k;
            c[k] = i < p.blocks ? row[i] : 0;
            sum += c[k];
        }
        int32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        int32_t at = carry + inc - sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + lane * 4 + k;
            if (i < p.blocks) row[i] = at;
            at += c[k];
        }
        carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) p.table[(int64_t)p.experts * p.blocks + e] = carry;
}

// Ranks within blocks become rows.
__global__ void __launch_bounds__(256) route_place_kernel(const RouteParams p) {
    pdl_enter();
    __shared__ int32_t s_first[kMaxExperts + 1];
    const int32_t *totals = p.table + (int64_t)p.experts * p.blocks;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s_first[e] = totals[e];
    __syncthreads();
    block_scan<256>(s_first, p.experts);
    const int64_t pairs = (int64_t)p.tokens * p.top_k;
    const int64_t lo = (int64_t)blockIdx.x * kChunkTokens * p.top_k;
    for (int64_t i = lo + threadIdx.x; i < lo + kChunkTokens * p.top_k && i < pairs; i += blockDim.x) {
        const int e = p.indices[i];
        if (e >= 0) {
            const int32_t slot = s_first[e] + p.table[(int64_t)e * p.blocks + blockIdx.x] + p.slots[i];
            p.slots[i] = slot;
            p.order[slot] = (int32_t)i;
        }
        if (i >= s_first[p.experts]) p.order[i] = -1;
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) p.offsets[e] = s_first[e];
}

template <typename T, int EPL>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteParams p) {
    pdl_enter();
    __shared__ float s_ds[8][EPL * 32];             // a token's scores' gradient, by expert
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= p.tokens) return;
    float *row = s_ds[threadIdx.x >> 5];
    float x[EPL], s[EPL];
    const T *logits = static_cast<const T *>(p.logits) + (int64_t)t * p.ldl;
    load_row<T, EPL>(logits, p.experts, lane, p.wide, x);
    int mine = lane < p.top_k ? p.indices[(int64_t)t * p.top_k + lane] : -1;
    if (mine >= p.experts) mine = -1;
    float g = mine >= 0 ? p.scale * p.grad[(int64_t)t * p.top_k + lane] : 0.f;
    float m = 0.f, z = 1.f, sel = mine >= 0 ? OpType<T>::up(logits[mine]) : -INFINITY;
    if (p.score == GEMM_SCORE_SOFTMAX) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) m = fmaxf(m, x[i]);
        m = warp_max(m);
        z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            s[i] = softmax_term(x[i], m);
            z += s[i];
        }
        z = warp_sum(z);
        const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] *= inv;
    }
#pragma unroll
    for (int i = 0; i < EPL; i += 4)
        *reinterpret_cast<float4 *>(row + expert_of(i, lane)) = make_float4(0.f, 0.f, 0.f, 0.f);
    sel = score_of(p.score, sel, m, z);
    if (p.renormalize) {
        // with the weights themselves, so that one chosen expert's (always 1) gives exactly 0
        const float sum = warp_sum(sel);
        if (sum > 0.f) g = (g - warp_sum(g * (sel / sum))) / sum;
    }
    if (mine < 0) g = 0.f;
    const float sum = warp_sum(g * sel);
    __syncwarp();
    if (mine >= 0) row[mine] = g;
    __syncwarp();
    float ds[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(row + expert_of(i, lane));
        ds[i] = v.x;
        ds[i + 1] = v.y;
        ds[i + 2] = v.z;
        ds[i + 3] = v.w;
    }
    if (p.score == GEMM_SCORE_SIGMOID) {
        // s (1 - s), for the chosen experts only.  1 - s is the sigmoid of -x: from the
        // rounded s it would lose its digits as x grows, and be 0 from x = 17 on.
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            s[i] = ds[i] != 0.f ? score_of(p.score, x[i], m, z) * (1.f / (1.f + expf(x[i]))) : 0.f;
    }
    T *out = static_cast<T *>(p.dlogits) + (int64_t)t * p.ldd;
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const int e = expert_of(i, lane);
        struct alignas(4 * sizeof(T)) V4 { T v[4]; } v;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float d = p.score == GEMM_SCORE_SIGMOID ? ds[i + k] * s[i + k] : s[i + k] * (ds[i + k] - sum);
            v.v[k] = OpType<T>::down(d);
        }
        if (p.d_wide && e < p.experts) {
            *reinterpret_cast<V4 *>(out + e) = v;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k < p.experts) out[e + k] = v.v[k];
        }
    }
}

int check_route(int64_t tokens, int64_t experts, int type, int64_t ldl, const gemm_route_t *how) {
    if (!op_type_ok(type)) return api_error(GEMM_ERR_INVALID_ARG, "unknown element type");
    if (!how) return api_error(GEMM_ERR_INVALID_ARG, "how is NULL");
    if (tokens < 0 || tokens > 0x7fffffffLL - 64) return api_error(GEMM_ERR_INVALID_ARG, "tokens out of range");
    if (experts < 1 || experts > kMaxExperts)
        return api_error(GEMM_ERR_INVALID_ARG, "experts must be in [1, 1024]");
    if (!op_read_pitch_ok(ldl, experts)) return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    if (how->score != GEMM_SCORE_SOFTMAX && how->score != GEMM_SCORE_SIGMOID)
        return api_error(GEMM_ERR_INVALID_ARG, "unknown score");
    if (how->group_score != GEMM_GROUP_MAX && how->group_score != GEMM_GROUP_TOP2)
        return api_error(GEMM_ERR_INVALID_ARG, "unknown group score");
    if (how->groups < 1 || how->groups > kMaxGroups || experts % how->groups != 0)
        return api_error(GEMM_ERR_INVALID_ARG, "groups must be in [1, 32] and divide experts");
    if (how->top_groups < 1 || how->top_groups > how->groups)
        return api_error(GEMM_ERR_INVALID_ARG, "top_groups must be in [1, groups]");
    if (how->top_k < 1 || how->top_k > kMaxTopK || how->top_k > how->top_groups * (experts / how->groups))
        return api_error(GEMM_ERR_INVALID_ARG, "top_k must be in [1, 32] and at most the experts of top_groups groups");
    if (tokens * how->top_k > 0x7fffffffLL) return api_error(GEMM_ERR_INVALID_ARG, "tokens * top_k must be below 2^31");
    return GEMM_OK;
}

RouteParams route_params(int64_t tokens, int64_t experts, int type, const void *logits, int64_t ldl,
                         const gemm_route_t *how) {
    RouteParams p = {};
    p.logits = logits;
    p.ldl = ldl;
    p.tokens = (int)tokens;
    p.experts = (int)experts;
    p.top_k = how->top_k;
    p.score = how->score;
    p.groups = how->groups;
    p.per = (int)experts / how->groups;
    p.top_groups = how->top_groups;
    p.top2 = how->group_score == GEMM_GROUP_TOP2;
    p.renormalize = how->renormalize != 0;
    p.scale = how->scale;
    p.wide = experts % 4 == 0 && op_wide(logits, ldl, op_type_bytes(type));
    return p;
}

// Calls f with the experts a lane holds as an integral constant.
template <typename F> cudaError_t by_experts(int experts, F &&f) {
    if (experts <= 128) return f(std::integral_constant<int, 4>{});
    if (experts <= 256) return f(std::integral_constant<int, 8>{});
    if (experts <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

}  // namespace
}  // namespace tcgemm

using namespace tcgemm;

extern "C" {

int gemm_route(int64_t tokens, int64_t experts, int type, const void *logits, int64_t ldl, const float *bias,
               const gemm_route_t *how, int32_t *indices, float *weights, int32_t *offsets, int32_t *order,
               int32_t *slots, struct CUstream_st *stream_) {
    api_clear_error();
    int rc = check_route(tokens, experts, type, ldl, how);
    if (rc) return rc;
    const bool ordered = offsets || order || slots;
    if (ordered && (!offsets || (tokens > 0 && (!order || !slots))))
        return api_error(GEMM_ERR_INVALID_ARG, "offsets, order and slots are all given or all NULL");
    const int eb = op_type_bytes(type);
    const uint64_t pairs = (uint64_t)(tokens * how->top_k) * 4;
    OpSpan spans[] = {{"logits", logits, op_extent(tokens, experts, ldl, eb), eb, false},
                            {"bias", bias, bias && tokens > 0 ? (uint64_t)experts * 4 : 0, 4, false},
                            {"indices", indices, pairs, 4, true},
                            {"weights", weights, pairs, 4, true},
                            {"offsets", offsets, ordered ? (uint64_t)(experts + 1) * 4 : 0, 4, true},
                            {"order", order, ordered ? pairs : 0, 4, true},
                            {"slots", slots, ordered ? pairs : 0, 4, true}};
    if (tokens == 0 && !ordered) return GEMM_OK;
    if ((rc = op_check(spans, 7, nullptr))) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (tokens == 0)
        return op_launched("offsets of no tokens", cudaMemsetAsync(offsets, 0, (size_t)(experts + 1) * 4, stream));

    RouteParams p = route_params(tokens, experts, type, logits, ldl, how);
    p.bias = bias;
    p.indices = indices;
    p.weights = weights;
    p.offsets = offsets;
    p.order = order;
    p.slots = slots;
    const bool grouped = p.groups > 1 && p.top_groups < p.groups;
    if (tokens <= kClusterTokens && ordered) {
        const cudaError_t e = op_by_type(type, [&](auto t) {
            return by_experts(p.experts, [&](auto epl) {
                constexpr int EPL = decltype(epl)::value;
                auto kern = route_cluster_kernel<decltype(t), EPL>;
                const size_t smem = grouped ? kWarps * EPL * 33 * 4 : 0;
                cudaError_t f = cudaSuccess;
                if (smem > 32 * 1024) f = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
                if (f != cudaSuccess) return f;
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3((unsigned)((p.tokens + kWarps - 1) / kWarps));
                cfg.blockDim = dim3(kWarps * 32);
                cfg.dynamicSmemBytes = smem;
                cfg.stream = stream;
                cudaLaunchAttribute attr[2];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = cfg.gridDim.x;
                attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
                attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
                attr[1].val.programmaticStreamSerializationAllowed = 1;
                cfg.attrs = attr;
                cfg.numAttrs = options_snapshot().pdl != 1 ? 2 : 1;
                return cudaLaunchKernelEx(&cfg, kern, p);
            });
        });
        return op_launched("route launch", e);
    }
    p.blocks = (p.tokens + kChunkTokens - 1) / kChunkTokens;
    void *ws = nullptr;
    if (ordered) {
        const size_t bytes = ((size_t)p.experts * p.blocks + p.experts) * 4;
        int dev = 0;
        cudaGetDevice(&dev);
        const cudaError_t e = op_malloc(&ws, bytes, dev, stream);
        if (e != cudaSuccess) {
            cudaGetLastError();
            char msg[128];
            std::snprintf(msg, sizeof msg, "workspace of %zu bytes: %s", bytes, cudaGetErrorString(e));
            return api_error(GEMM_ERR_NO_MEMORY, msg);
        }
        p.table = static_cast<int32_t *>(ws);
    }
    cudaError_t e = op_by_type(type, [&](auto t) {
        return by_experts(p.experts, [&](auto epl) {
            constexpr int EPL = decltype(epl)::value;
            auto kern = route_kernel<decltype(t), EPL>;
            const size_t smem = grouped ? kWarps * EPL * 33 * 4 : 0;
            cudaError_t f = cudaSuccess;
            if (smem > 32 * 1024) f = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (f != cudaSuccess) return f;
            return launch_pdl(kern, dim3(p.blocks), dim3(kWarps * 32), smem, stream, p);
        });
    });
    if (ordered) {
        if (e == cudaSuccess) e = launch_pdl(route_scan_kernel, dim3((p.experts + 3) / 4), dim3(128), 0, stream, p);
        if (e == cudaSuccess)
            e = launch_pdl(route_place_kernel, dim3(p.blocks), dim3(256), 0, stream, p);
        const cudaError_t f = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess) e = f;
    }
    return op_launched("route launch", e);
}

int gemm_route_backward(int64_t tokens, int64_t experts, int type, const void *logits, int64_t ldl,
                        const gemm_route_t *how, const int32_t *indices, const float *grad, void *dlogits, int64_t ldd,
                        struct CUstream_st *stream_) {
    api_clear_error();
    int rc = check_route(tokens, experts, type, ldl, how);
    if (rc) return rc;
    if (ldd < experts || ldd > (1LL << 36)) return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    if (tokens == 0) return GEMM_OK;
    const int eb = op_type_bytes(type);
    const uint64_t pairs = (uint64_t)(tokens * how->top_k) * 4;
    OpSpan spans[] = {{"logits", logits, op_extent(tokens, experts, ldl, eb), eb, false},
                            {"indices", indices, pairs, 4, false},
                            {"grad", grad, pairs, 4, false},
                            {"dlogits", dlogits, op_extent(tokens, experts, ldd, eb), eb, true}};
    if ((rc = op_check(spans, 4, nullptr))) return rc;
    RouteParams p = route_params(tokens, experts, type, logits, ldl, how);
    p.indices = const_cast<int32_t *>(indices);
    p.grad = grad;
    p.dlogits = dlogits;
    p.ldd = ldd;
    p.d_wide = experts % 4 == 0 && op_wide(dlogits, ldd, eb);
    const cudaError_t e = op_by_type(type, [&](auto t) {
        return by_experts(p.experts, [&](auto epl) {
            return launch_pdl(route_backward_kernel<decltype(t), decltype(epl)::value>, dim3((p.tokens + 7) / 8),
                              dim3(256), 0, reinterpret_cast<cudaStream_t>(stream_), p);
        });
    });
    return op_launched("route backward launch", e);
}

}  // extern "C"

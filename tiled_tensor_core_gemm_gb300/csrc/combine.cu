// The weighted combination of the experts' rows and its gradients.
//
//   out[t]       = sum_j w[t][j] * Y[slot(t, j)]      (FP32, in the order of j, rounded once)
//   dY[slot]     = w[t][j] * g[t]
//   dw[t][j]     = <g[t], Y[slot]>
//
// Both are one pass over the rows and bound by HBM.  A block takes one token:
// its threads walk the hidden dimension eight elements (16 or 32 bytes) at a
// time, all top_k rows' loads of a step in flight together.  In the backward
// pass g[t] is read once and each row's product with it is kept per thread,
// then summed over the block in a fixed order, so results do not depend on
// timing.
#include "ops.h"

namespace tcgemm {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kChunk = 8;     // rows of a token taken together

struct CombineParams {
    const void *Y, *grad;
    int64_t ldy, ldg, ldo, hidden, rows;
    const int32_t *slots, *order;
    const float *weights;
    void *out;                // out (forward) or dY (backward)
    float *dweights;
    int top_k;
    int wide;                 // every row of every array starts on 16 bytes
};

template <typename T>
__global__ void __launch_bounds__(kMaxThreads) combine_kernel(const CombineParams p) {
    pdl_enter();
    const int64_t t = blockIdx.x;
    const int64_t h = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 8;
    if (h >= p.hidden) return;
    const int have = (int)(p.hidden - h < 8 ? p.hidden - h : 8);
    const T *Y = static_cast<const T *>(p.Y);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < p.top_k; j0 += kChunk) {
        OpVec8<T> y[kChunk];
        float w[kChunk];
        bool real[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const bool in = j0 + j < p.top_k;
            const int64_t s = in ? p.slots[t * p.top_k + j0 + j] : -1;
            real[j] = s >= 0 && s < p.rows;
            w[j] = !real[j] ? 0.f : p.weights ? p.weights[t * p.top_k + j0 + j] : 1.f;
            if (real[j]) y[j] = op_load8<T>(Y + s * p.ldy + h, have, p.wide);
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
            if (real[j]) {
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[j], OpType<T>::up(y[j].v[k]), acc[k]);
            }
    }
    OpVec8<T> o;
#pragma unroll
    for (int k = 0; k < 8; ++k) o.v[k] = OpType<T>::down(acc[k]);
    op_store8<T>(static_cast<T *>(p.out) + t * p.ldo + h, o, have, p.wide);
}

template <typename T>
__global__ void __launch_bounds__(kMaxThreads) combine_backward_kernel(const CombineParams p) {
    pdl_enter();
    __shared__ float s_part[kMaxThreads / 32][kChunk];
    const int64_t t = blockIdx.x;
    const T *Y = static_cast<const T *>(p.Y), *G = static_cast<const T *>(p.grad) + t * p.ldg;
    T *D = static_cast<T *>(p.out);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < p.top_k; j0 += kChunk) {
        float w[kChunk], dot[kChunk];
        int64_t s[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const bool in = j0 + j < p.top_k;
            const int64_t at = in ? p.slots[t * p.top_k + j0 + j] : -1;
            s[j] = at >= 0 && at < p.rows ? at : -1;
            w[j] = s[j] >= 0 ? p.weights[t * p.top_k + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int64_t h = (int64_t)threadIdx.x * 8; h < p.hidden; h += (int64_t)blockDim.x * 8) {
            const int have = (int)(p.hidden - h < 8 ? p.hidden - h : 8);
            const OpVec8<T> g = op_load8<T>(G + h, have, p.wide);
            OpVec8<T> y[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
                if (s[j] >= 0) y[j] = op_load8<T>(Y + s[j] * p.ldy + h, have, p.wide);
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
                if (s[j] >= 0) {
                    OpVec8<T> d;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float gk = OpType<T>::up(g.v[k]);
                        d.v[k] = OpType<T>::down(w[j] * gk);
                        dot[j] = fmaf(gk, OpType<T>::up(y[j].v[k]), dot[j]);
                    }
                    op_store8<T>(D + s[j] * p.ldo + h, d, have, p.wide);
                }
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
            if (lane == 0) s_part[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kChunk && j0 + (int)threadIdx.x < p.top_k) {
            float sum = 0.f;
            for (int i = 0; i < warps; ++i) sum += s_part[i][threadIdx.x];
            p.dweights[t * p.top_k + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
    // rows past the experts' last: no token's, so their gradient is zero
    if (p.order) {
        for (int j = 0; j < p.top_k; ++j) {
            const int64_t r = t * p.top_k + j;
            if (r >= p.rows || p.order[r] >= 0) continue;
            OpVec8<T> z;
#pragma unroll
            for (int k = 0; k < 8; ++k) z.v[k] = OpType<T>::down(0.f);
            for (int64_t h = (int64_t)threadIdx.x * 8; h < p.hidden; h += (int64_t)blockDim.x * 8)
                op_store8<T>(D + r * p.ldo + h, z, (int)(p.hidden - h < 8 ? p.hidden - h : 8), p.wide);
        }
    }
}

int check_sizes(int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows, int type) {
    if (!op_type_ok(type)) return api_error(GEMM_ERR_INVALID_ARG, "unknown element type");
    const int64_t kMax = 0x7fffffffLL;
    if (tokens < 0 || hidden < 0 || rows < 0 || tokens > kMax || hidden > kMax || rows > kMax)
        return api_error(GEMM_ERR_INVALID_ARG, "size out of range (0 <= sizes < 2^31)");
    if (top_k < 1 || top_k > 1024 || tokens * top_k > kMax)
        return api_error(GEMM_ERR_INVALID_ARG, "top_k out of range");
    return GEMM_OK;
}

// Threads that cover `hidden` in steps of eight, a whole number of warps.
int threads_for(int64_t hidden) {
    const int64_t want = ((hidden + 7) / 8 + 31) / 32 * 32;
    return (int)(want < 32 ? 32 : want < kMaxThreads ? want : kMaxThreads);
}

}  // namespace
}  // namespace tcgemm

using namespace tcgemm;

extern "C" {

int gemm_combine(int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows, int type, const void *Y, int64_t ldy,
                 const int32_t *slots, const float *weights, void *out, int64_t ldo, struct CUstream_st *stream_) {
    api_clear_error();
    int rc = check_sizes(tokens, top_k, hidden, rows, type);
    if (rc) return rc;
    const int64_t kLdMax = 1LL << 36;
    if (ldy < hidden || ldo < hidden || ldy > kLdMax || ldo > kLdMax)
        return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    if (tokens == 0 || hidden == 0) return GEMM_OK;
    const int eb = op_type_bytes(type);
    const OpSpan spans[] = {{"Y", Y, op_extent(rows, hidden, ldy, eb), eb, false},
                            {"slots", slots, (uint64_t)(tokens * top_k) * 4, 4, false},
                            {"weights", weights, weights ? (uint64_t)(tokens * top_k) * 4 : 0, 4, false},
                            {"out", out, op_extent(tokens, hidden, ldo, eb), eb, true}};
    if ((rc = op_check(spans, 4, nullptr))) return rc;
    CombineParams p = {};
    p.Y = Y;
    p.ldy = ldy;
    p.slots = slots;
    p.weights = weights;
    p.out = out;
    p.ldo = ldo;
    p.hidden = hidden;
    p.rows = rows;
    p.top_k = (int)top_k;
    p.wide = op_wide(Y, ldy, eb) && op_wide(out, ldo, eb);
    const int threads = threads_for(hidden);
    const dim3 grid((unsigned)tokens, (unsigned)((hidden + threads * 8 - 1) / (threads * 8)), 1);
    if (grid.y > 65535) return api_error(GEMM_ERR_INVALID_ARG, "hidden out of range");
    const cudaError_t e = op_by_type(type, [&](auto t) {
        return launch_pdl(combine_kernel<decltype(t)>, grid, dim3(threads), 0,
                          reinterpret_cast<cudaStream_t>(stream_), p);
    });
    return op_launched("combine launch", e);
}

int gemm_combine_backward(int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows, int type, const void *grad,
                          int64_t ldg, const void *Y, int64_t ldy, const int32_t *slots, const float *weights,
                          const int32_t *order, void *dY, int64_t ldd, float *dweights, struct CUstream_st *stream_) {
    api_clear_error();
    int rc = check_sizes(tokens, top_k, hidden, rows, type);
    if (rc) return rc;
    const int64_t kLdMax = 1LL << 36;
    if (ldg < hidden || ldy < hidden || ldd < hidden || ldg > kLdMax || ldy > kLdMax || ldd > kLdMax)
        return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    if (order && rows != tokens * top_k)
        return api_error(GEMM_ERR_INVALID_ARG, "order needs rows = tokens * top_k");
    if (tokens == 0) return GEMM_OK;
    const int eb = op_type_bytes(type);
    const uint64_t pairs = (uint64_t)(tokens * top_k) * 4;
    const OpSpan spans[] = {{"grad", grad, op_extent(tokens, hidden, ldg, eb), eb, false},
                            {"Y", Y, op_extent(rows, hidden, ldy, eb), eb, false},
                            {"slots", slots, pairs, 4, false},
                            {"weights", weights, pairs, 4, false},
                            {"order", order, order ? pairs : 0, 4, false},
                            {"dY", dY, op_extent(rows, hidden, ldd, eb), eb, true},
                            {"dweights", dweights, pairs, 4, true}};
    if ((rc = op_check(spans, 7, nullptr))) return rc;
    CombineParams p = {};
    p.Y = Y;
    p.ldy = ldy;
    p.grad = grad;
    p.ldg = ldg;
    p.slots = slots;
    p.order = order;
    p.weights = weights;
    p.out = dY;
    p.ldo = ldd;
    p.dweights = dweights;
    p.hidden = hidden;
    p.rows = rows;
    p.top_k = (int)top_k;
    p.wide = op_wide(Y, ldy, eb) && op_wide(grad, ldg, eb) && op_wide(dY, ldd, eb);
    const cudaError_t e = op_by_type(type, [&](auto t) {
        return launch_pdl(combine_backward_kernel<decltype(t)>, dim3((unsigned)tokens), dim3(threads_for(hidden)), 0,
                          reinterpret_cast<cudaStream_t>(stream_), p);
    });
    return op_launched("combine backward launch", e);
}

}  // extern "C"
